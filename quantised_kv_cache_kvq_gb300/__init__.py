"""GB300 quantised KV cache: packed KIVI / INT8 / FP8 caches, single-query decode attention
over them and what speculative decoding needs next to it (attention of drafted tokens over
a cache, reading a cache back, rotary positions), in CUDA kernels behind the C ABI of
include/kvq.h.

`QuantizedKVCache` is a convenience holder: it allocates the cache and the decode
workspace as torch device tensors (torch serves only as the device allocator and stream
source) and forwards every call to libkvq.so.
"""
import math

from ._native import (  # noqa: F401
    EXPORTS, KVQ_BYTES_FORMULA, KVQ_BYTES_LAYOUT, KVQ_DTYPE_BF16, KVQ_DTYPE_F32,
    KVQ_NO_AUTOFLUSH, KVQ_SCHEME_FP8_E4M3, KVQ_SCHEME_FP8_E5M2, KVQ_SCHEME_INT4, KVQ_SCHEME_INT8,
    KVQ_SCHEME_KIVI,
    KVQ_STATUS_BAD_PAGE, KVQ_STATUS_CAPACITY, KVQ_STATUS_NONFINITE, KVQ_STATUS_RING_FULL, KVQ_STATUS_TIMEOUT,
    KVQ_MAX_ROTARY_DIM, KVQ_MAX_TREE_NODES, KVQ_ROPE_HALF, KVQ_ROPE_INTERLEAVED, KVQ_ROPE_SCALE_BY_PARTS,
    KVQ_ROPE_SCALE_LINEAR, KVQ_ROPE_SCALE_NONE, KVQ_ROPE_SCALE_NTK, KVQ_ROPE_TRANSPOSE,
    KvqConfig, KvqError, KvqRopeConfig, kvq_cache_bytes, kvq_cache_init, kvq_decode_attention,
    kvq_decode_attention_noalloc,
    kvq_flush_group, kvq_quantize_append, kvq_read_status, kvq_read_tokens, kvq_rope, kvq_rope_frequencies,
    kvq_sequence_lengths, kvq_tree_attention, kvq_tree_workspace_bytes, kvq_workspace_bytes, library_path, load, status_string,
)

_SCHEMES = {"kivi": KVQ_SCHEME_KIVI, "int8": KVQ_SCHEME_INT8, "fp8": KVQ_SCHEME_FP8_E4M3,
            "fp8e5m2": KVQ_SCHEME_FP8_E5M2, "int4": KVQ_SCHEME_INT4}


def make_config(scheme, layers, batch, q_heads, kv_heads, head_dim, max_tokens, bits=None,
                group_k=32, group_v=32, residual=0, in_dtype="bf16", page_groups=0, num_pages=0,
                block_table=None, rope_base=0.0, outliers=0) -> KvqConfig:
    """block_table: paged KIVI layout, a device int32 tensor [batch][max_pages]; rope_base:
    KIVI keys cached before the rotary embedding (its base; 0 for keys cached as given);
    outliers: KIVI dense-and-sparse, elements per quantisation vector kept aside in bf16."""
    s = _SCHEMES[scheme] if isinstance(scheme, str) else int(scheme)
    if bits is None:
        bits = {KVQ_SCHEME_KIVI: 2, KVQ_SCHEME_INT4: 4}.get(s, 8)
    c = KvqConfig()
    c.scheme, c.layers, c.batch, c.q_heads, c.kv_heads = s, layers, batch, q_heads, kv_heads
    c.head_dim, c.bits, c.group_k, c.group_v, c.residual = head_dim, bits, group_k, group_v, residual
    c.max_tokens = max_tokens
    c.in_dtype = KVQ_DTYPE_BF16 if in_dtype in ("bf16", KVQ_DTYPE_BF16) else KVQ_DTYPE_F32
    c.page_groups, c.num_pages = page_groups, num_pages
    c.rope_base = float(rope_base)
    c.outliers = int(outliers)
    c.set_block_table(block_table)
    return c


def max_pages(cfg) -> int:
    """Block-table entries per sequence of a paged configuration."""
    ng = (cfg.max_tokens - cfg.residual) // cfg.group_k if cfg.max_tokens > cfg.residual else 0
    return (ng + cfg.page_groups - 1) // cfg.page_groups if cfg.page_groups > 0 else 0


def _fits(x, shape, dtype, device):
    """Whether the library reads tensor x rightly: a contiguous tensor of this shape and type on
    this device, or in page-locked host memory."""
    return (x.shape == shape and x.dtype == dtype and x.is_contiguous()
            and (x.device == device or not x.is_cuda and (x.numel() == 0 or x.is_pinned())))


def _expect(name, x, shape, dtype, device):
    """Refuses a tensor that the library would read wrongly."""
    if not _fits(x, shape, dtype, device):
        raise ValueError("%s: expected a contiguous %s tensor of shape %s on %s (or page-locked), got %s %s on %s%s" % (
            name, dtype, tuple(shape), device, x.dtype, tuple(x.shape), x.device,
            "" if x.is_contiguous() else ", not contiguous"))


class _on:
    """torch.cuda.device, where the device is not the current one already."""

    def __init__(self, device):
        self.device, self.guard = device, None

    def __enter__(self):
        import torch
        if torch.cuda.current_device() != self.device.index:
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()

    def __exit__(self, *e):
        if self.guard is not None:
            self.guard.__exit__(*e)


class QuantizedKVCache:
    """A cache and its decode workspace on one GPU."""

    def __init__(self, cfg: KvqConfig, device="cuda"):
        import torch
        load()
        self.cfg = cfg
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.nbytes = kvq_cache_bytes(cfg, cfg.max_tokens, KVQ_BYTES_LAYOUT)
        self.cache = torch.empty(self.nbytes, dtype=torch.uint8, device=self.device)
        kvq_cache_init(cfg, self.cache)
        self.workspace = torch.zeros(kvq_workspace_bytes(cfg), dtype=torch.uint8, device=self.device)
        self._tree_workspaces = {}

    def append(self, layer, k_new, v_new, seq_begin=0, n_valid=None, fp8_scales=None, flags=0,
               stream=None):
        """k_new, v_new: [seq_count][n_new][kv_heads][head_dim] device tensors."""
        seq_count, n_new = k_new.shape[0], k_new.shape[1]
        kvq_quantize_append(self.cfg, self.cache, layer, seq_begin, seq_count, k_new, v_new, n_new,
                            n_valid, fp8_scales, flags, stream)

    def flush(self, layer, stream=None):
        kvq_flush_group(self.cfg, self.cache, layer, stream)

    def decode(self, layer, q, softmax_scale=None, out=None, stream=None):
        import torch
        if softmax_scale is None:
            softmax_scale = 1.0 / math.sqrt(self.cfg.head_dim)
        if out is None:
            out = torch.empty(self.cfg.batch, self.cfg.q_heads, self.cfg.head_dim,
                              dtype=torch.float32, device=self.device)
        kvq_decode_attention(self.cfg, self.cache, layer, q, softmax_scale, out, self.workspace,
                             stream=stream)
        return out

    def tree_workspace(self, nodes):
        """Scratch for tree_decode calls of up to `nodes` drafts: one per set of calls that may
        overlap on the GPU (and one per CUDA graph that may be replayed beside another)."""
        import torch
        return torch.zeros(kvq_tree_workspace_bytes(self.cfg, nodes), dtype=torch.uint8, device=self.device)

    def tree_decode(self, layer, q, k_draft, v_draft, mask=None, n_nodes=None, softmax_scale=None, out=None,
                    workspace=None, stream=None):
        """Attention of drafted tokens over the cached tokens and the drafts that they see.
        q: bf16 [batch][nodes][q_heads][head_dim]; k_draft, v_draft: bf16 [batch][nodes]
        [kv_heads][head_dim]; mask: bool or uint8 [batch][nodes][nodes] (None: a chain);
        n_nodes: int32 [batch] or None.  Returns bf16 [batch][nodes][q_heads][head_dim].
        workspace: tree_workspace(nodes), by default one that the cache keeps for each number
        of nodes (calls on several streams, and graphs replayed side by side, need their own)."""
        import torch
        c, device, bf16 = self.cfg, self.device, torch.bfloat16
        batch, heads, D = c.batch, c.kv_heads, c.head_dim
        nodes = q.shape[1] if q.dim() == 4 else 0
        _expect("q", q, (batch, nodes, c.q_heads, D), bf16, device)
        _expect("k_draft", k_draft, (batch, nodes, heads, D), bf16, device)
        _expect("v_draft", v_draft, (batch, nodes, heads, D), bf16, device)
        if mask is not None:
            _expect("mask", mask, (batch, nodes, nodes), torch.uint8 if mask.dtype == torch.uint8 else torch.bool, device)
        if n_nodes is not None:
            _expect("n_nodes", n_nodes, (batch,), torch.int32, device)
        with _on(device):
            if workspace is None:
                workspace = self._tree_workspaces.get(nodes)
                if workspace is None:
                    if torch.cuda.is_current_stream_capturing():    # (it would be the graph's memory)
                        raise ValueError("tree_decode: a captured call needs a workspace made before the capture")
                    workspace = self._tree_workspaces[nodes] = self.tree_workspace(nodes)
            if out is None:
                out = torch.empty(q.shape, dtype=bf16, device=device)
            else:
                _expect("out", out, q.shape, bf16, device)
            kvq_tree_attention(c, self.cache, layer, nodes, q, k_draft, v_draft, mask, n_nodes,
                               1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale, out, workspace,
                               stream=stream)
        return out

    def read(self, layer, first=0, count=None, seq_begin=0, seq_count=None, dtype="bf16", k_out=None, v_out=None,
             stream=None):
        """Cached tokens [first, first + count) of sequences [seq_begin, seq_begin + seq_count),
        dequantised: (keys, values) [seq_count][count][kv_heads][head_dim], bf16 or f32; rows
        past a sequence's tokens are 0.  first: a number, or a device int32 tensor [seq_count];
        count: by default up to the capacity."""
        import torch
        c = self.cfg
        starts = first if isinstance(first, torch.Tensor) else None
        if seq_count is None:
            seq_count = c.batch - seq_begin
        if starts is not None:
            _expect("first", starts, (seq_count,), torch.int32, self.device)
            first = 0
        if count is None:
            count = c.max_tokens - first
        code = {"bf16": KVQ_DTYPE_BF16, "f32": KVQ_DTYPE_F32}[dtype]
        kind = torch.float32 if code == KVQ_DTYPE_F32 else torch.bfloat16
        shape = (seq_count, count, c.kv_heads, c.head_dim)
        with _on(self.device):
            outs = [torch.empty(shape, dtype=kind, device=self.device) if x is None else x for x in (k_out, v_out)]
            _expect("k_out", outs[0], shape, kind, self.device)
            _expect("v_out", outs[1], shape, kind, self.device)
            kvq_read_tokens(c, self.cache, layer, seq_begin, seq_count, starts, first, count, outs[0], outs[1], code,
                            stream)
        return outs[0], outs[1]

    def status(self, stream=None):
        word = kvq_read_status(self.cache, self.workspace, stream)
        for ws in self._tree_workspaces.values():
            word |= kvq_read_status(None, ws, stream)
        return word

    def lengths(self, layer, stream=None):
        import torch
        n = torch.empty(self.cfg.batch, dtype=torch.int32, device=self.device)
        qn = torch.empty(self.cfg.batch, dtype=torch.int32, device=self.device)
        kvq_sequence_lengths(self.cfg, self.cache, layer, n, qn, stream)
        return n, qn


_ROPE_LAYOUTS = {"half": KVQ_ROPE_HALF, "interleaved": KVQ_ROPE_INTERLEAVED}
_ROPE_SCALINGS = {"none": KVQ_ROPE_SCALE_NONE, "linear": KVQ_ROPE_SCALE_LINEAR, "ntk": KVQ_ROPE_SCALE_NTK,
                  "by_parts": KVQ_ROPE_SCALE_BY_PARTS}


class RotaryEmbedding:
    """Rotary positions of queries and keys (kvq_rope_config names the parameters; the
    frequencies are computed once, here).  For a cache with rope_base the queries and the
    drafts' keys are turned with the same base, all of a head, layout "half"."""

    def __init__(self, head_dim, base=10000.0, rotary_dim=None, layout="half", scaling="none", factor=1.0, low=1.0,
                 high=4.0, original_context=8192, magnitude=1.0):
        self.rope = KvqRopeConfig(
            head_dim=head_dim, rotary_dim=head_dim if rotary_dim is None else rotary_dim, layout=_ROPE_LAYOUTS[layout],
            dtype=KVQ_DTYPE_BF16, scaling=_ROPE_SCALINGS[scaling], original_context=original_context, base=base,
            factor=factor, low=low, high=high, magnitude=magnitude)
        self.frequencies = kvq_rope_frequencies(self.rope)
        self._f32 = KvqRopeConfig.from_buffer_copy(self.rope)
        self._f32.dtype = KVQ_DTYPE_F32

    def rotate(self, q, k, positions, q_out=None, k_out=None, transpose=False, stream=None):
        """q, k: [tokens][heads][head_dim], bf16 or float32 (one of them may be None), each
        token's heads one after another, the tokens at any stride (slices of a fused
        projection); positions: int32 [tokens].  Returns (q, k) turned, in new tensors or in
        q_out, k_out (q and k themselves: in place).  transpose: the gradient."""
        import torch
        x = k if q is None else q
        if x is None or x.dim() != 3 or x.dtype not in (torch.bfloat16, torch.float32) or not x.is_cuda:
            raise ValueError("rotate: expected bfloat16 or float32 rows [tokens][heads][head_dim] on a GPU")
        dtype, device, tokens = x.dtype, x.device, x.shape[0]
        _expect("positions", positions, (tokens,), torch.int32, device)
        with _on(device):
            if q is not None:
                q_out = self._rows("q", q, q_out, tokens, dtype, device)
                qa = (q, q_out, q.shape[1], q.stride(0), q_out.stride(0))
            else:
                qa, q_out = (None, None, 0, 0, 0), None
            if k is not None:
                k_out = self._rows("k", k, k_out, tokens, dtype, device)
                ka = (k, k_out, k.shape[1], k.stride(0), k_out.stride(0))
            else:
                ka, k_out = (None, None, 0, 0, 0), None
            kvq_rope(self.rope if dtype == torch.bfloat16 else self._f32, self.frequencies, positions, tokens, *qa, *ka,
                     KVQ_ROPE_TRANSPOSE if transpose else 0, stream)
        return q_out, k_out

    def _rows(self, name, x, y, tokens, dtype, device):
        """The output rows for input rows x; refuses what the library would read wrongly."""
        import torch
        D = self.rope.head_dim
        if y is None:
            y = torch.empty(x.shape, dtype=dtype, device=device)
        for z in (x, y):
            if z.dim() != 3 or z.shape != x.shape or z.shape[0] != tokens or z.shape[2] != D or z.dtype != dtype \
                    or z.device != device:
                raise ValueError("%s: expected %s [%d][heads][%d] on %s, got %s %s on %s" % (
                    name, dtype, tokens, D, device, z.dtype, tuple(z.shape), z.device))
            s = z.stride()
            if (s[2] != 1 and D > 1 or s[1] != D and z.shape[1] > 1) and z.numel():
                raise ValueError("%s: a token's heads must lie one after another" % name)
        return y
