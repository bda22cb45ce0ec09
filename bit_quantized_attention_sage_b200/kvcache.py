"""Rotary positions and the paged 8-bit key/value cache: ctypes wrappers of
``sage_rope*`` and ``sage_cache_*`` (include/sage.h documents the operators).

A streaming or serving loop keeps one ``KVCache8`` and, per step:

    k = rope(k, positions, inv_freq)                     # before it is cached
    cache_append(cache, k, v, pages, lengths)            # lengths: before
    lengths += n
    o, lse = cache_attn(rope(q, ...), cache, pages, lengths, "causal", return_lse=True)
    cache_weights(q, cache, lse, pages, lengths, "causal")     # optional:
    kept, lengths = cache_evict(cache, pages, lengths, keep)   # prune

Every call takes the tensors' device (not the current one) and, without
``stream``, that device's current stream; what it allocates belongs to that
stream.  Autograd sees rope alone: the cache's calls record no gradient.
"""
import ctypes
import functools
import math

PAGE = 64          # tokens per page
MIN_V_EXP = -40
_MASKS = "mask must be None, 'causal', ('block_causal', n) or " \
         "('window', frame_len, window_frames, sink_tokens)"


torch = None  # the module, once a call has brought a tensor (the package imports without it)
_TYPES = {}   # torch dtype -> type code
_Turn = None  # rope as an autograd function


def _load():
    global torch, _Turn
    import torch as t
    torch = t
    _TYPES.update({t.bfloat16: 0, t.float16: 1, t.float32: 2})

    class Turn(t.autograd.Function):
        @staticmethod
        def forward(ctx, x, positions, inv_freq, layout, amplitude, inverse):
            ctx.save_for_backward(positions, inv_freq)
            ctx.how = layout, amplitude, inverse
            return rope(x, positions, inv_freq, layout, amplitude, inverse)

        @staticmethod
        def backward(ctx, dy):
            layout, amplitude, inverse = ctx.how
            if dy.stride(-1) != 1:
                dy = dy.contiguous()
            return (rope(dy, *ctx.saved_tensors, layout, amplitude, not inverse),) + (None,) * 5

    _Turn = Turn


def _type(t):
    if torch is None:
        _load()
    return _TYPES.get(t.dtype, -1)


class _Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_i8", "k_scale", "v_f8", "v_exp", "weight")] + \
               [(n, ctypes.c_int) for n in ("n_pages", "heads", "D")]


class _Seqs(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("B", ctypes.c_int),
                ("max_pages", ctypes.c_int)]


class _Query(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_strides", ctypes.c_longlong * 3),
                ("q_lens", ctypes.c_void_p), ("type", ctypes.c_int), ("H", ctypes.c_int),
                ("Nq", ctypes.c_int), ("max_len", ctypes.c_int), ("scale", ctypes.c_float)]


_Strides = ctypes.c_longlong * 3


def declare(L):
    """Result and argument types of the library's functions (called by lib())."""
    global _L
    _L = L
    P, I, SZ, LL, F = (ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong,
                       ctypes.c_float)
    L.sage_rope.restype = I
    L.sage_rope.argtypes = [P, P, I, I, I, I, I, I, P, P, P, I, LL, P, F, I, I, P]
    L.sage_rope_tables.restype = I
    L.sage_rope_tables.argtypes = [I, I, P, I, P, F, P, P, P]
    L.sage_cache_append.restype = I
    L.sage_cache_append.argtypes = [P, P, P, P, I, I, P, P, P, P, P]
    L.sage_cache_read.restype = I
    L.sage_cache_read.argtypes = [P, P, I, P, P, P, P, P, P]
    L.sage_cache_attn_workspace_bytes.restype = SZ
    L.sage_cache_attn_workspace_bytes.argtypes = [I] * 10
    L.sage_cache_attn.restype = I
    L.sage_cache_attn.argtypes = [P, P, P, I, I, I, I, P, P, P, P, SZ, P]
    L.sage_cache_weights.restype = I
    L.sage_cache_weights.argtypes = [P, P, P, I, I, I, I, P, I, P]
    L.sage_cache_evict_workspace_bytes.restype = SZ
    L.sage_cache_evict_workspace_bytes.argtypes = [I] * 5
    L.sage_cache_evict.restype = I
    L.sage_cache_evict.argtypes = [P, P, I, I, I, P, I, P, P, P, SZ, P]


_L = None  # the library, once declare() has seen it


def _lib():
    if _L is None:
        from . import lib
        lib()
    return _L


def _check(code, what):
    if code != 0:
        from . import SageError
        raise SageError(code, what)


def _here(t, stream):
    """The current stream's handle if the call can run as it is: `t` on the
    current device, no other stream asked for.  None otherwise."""
    if torch is None:
        _load()
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    if stream is None and dev == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(dev)
    return None


class _There:
    """`t`'s device made current, and `stream` (or the device's current one):
    what is allocated inside belongs to that stream."""

    def __init__(self, t, stream):
        if torch is None:
            _load()
        if stream is not None and stream.device != t.device:
            raise ValueError("the stream belongs to %s, the tensors to %s" % (stream.device,
                                                                              t.device))
        self.device = torch.cuda.device(t.device)
        self.stream = torch.cuda.stream(stream)  # of None: no change

    def __enter__(self):
        self.device.__enter__()
        self.stream.__enter__()

    def __exit__(self, *exc):
        self.stream.__exit__(*exc)
        self.device.__exit__(*exc)


def _new(t):
    """An uninitialised contiguous tensor like `t`, and its strides."""
    out = torch.empty_like(t) if t.is_contiguous() else \
        torch.empty(t.shape, dtype=t.dtype, device=t.device)
    return out, _strides(out)


def _strides(t):
    b, h, n, c = t.stride()
    B, H, N, C = t.shape
    if c != 1 and C > 1:
        raise ValueError("the last dimension must have unit stride")
    return _Strides(b if B > 1 else 0, h if H > 1 else 0, n if N > 1 else 0)


def _out_strides(t):
    if 0 in t.stride() and any(t.shape[i] > 1 and t.stride(i) == 0 for i in range(3)):
        raise ValueError("out must not be an expanded tensor")
    return _strides(t)


def _meets(x, xs, y, ys, budget=2000):
    """Whether the output y, of x's shape, has memory in common with x in another
    way than being x: elements at the same places with the same strides (xs and
    ys, of _strides).  Such an output would overwrite inputs that other blocks
    have yet to read.  (True also where a search of `budget` steps does not
    tell.)"""
    es = x.element_size()
    B, H, N, D = x.shape
    away = y.data_ptr() - x.data_ptr()
    first = xs if away >= 0 else ys
    if abs(away) >= ((B - 1) * first[0] + (H - 1) * first[1] + (N - 1) * first[2] + D) * es or \
            away == 0 and xs[:] == ys[:]:
        return False
    # bytes from a run of D channels of x to one of y: away + the sum of
    # step * [lo .. hi] over the strides; the runs meet where that is within
    # D * es.  The largest stride first leaves a choice or two of each.
    reach = {}
    for strides, of_x in ((xs, True), (ys, False)):
        for s, n in zip(strides, x.shape):
            lo, hi = reach.get(s * es, (0, 0))
            reach[s * es] = (lo - n + 1, hi) if of_x else (lo, hi + n - 1)
    steps = sorted(((s, lo, hi) for s, (lo, hi) in reach.items() if s), reverse=True)
    rest = [(0, 0)]
    for s, lo, hi in reversed(steps):
        rest.insert(0, (rest[0][0] + s * lo, rest[0][1] + s * hi))

    def search(i, at):  # some sum of the steps from i on brings `at` within the run
        nonlocal budget
        budget -= 1
        low, high = at + rest[i][0], at + rest[i][1]
        if budget < 0 or low >= D * es or high <= -D * es:
            return budget < 0
        if i == len(steps):
            return True
        s, lo, hi = steps[i]
        a, b = rest[i + 1]
        k0 = max(lo, -((at + b + D * es - 1) // s))
        k1 = min(hi, (D * es - 1 - at - a) // s)
        return any(search(i + 1, at + s * k) for k in range(k0, k1 + 1))

    return search(0, away)


def _int32(t, shape, what, dev):
    if t.dtype is not torch.int32 or t.get_device() != dev or t.shape != shape or \
            not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor %s on cuda:%d" % (what, shape, dev))
    return t.data_ptr()


# ---------------------------------------------------------------- rotary positions

def rope_freqs(dim, theta=10000.0, scaling=None, device="cuda"):
    """Angle per position of the dim / 2 channel pairs (fp64 tensor on
    `device`) and the amplitude that goes with them.

    scaling: None: f_p = theta^(-2 p / dim).  ("linear", s): f_p / s.
    ("ntk", s): theta becomes theta s^(dim / (dim - 2)).  ("yarn", s, L[,
    fast, slow]): by parts -- pairs that turn `fast` (32) times or more within
    the original context L keep f_p, those below `slow` (1) turns get f_p / s,
    linear in the turns between; amplitude 0.1 ln s + 1."""
    import torch
    if dim < 2 or dim % 2:
        raise ValueError("dim must be even and at least 2")
    if not theta > 0:
        raise ValueError("theta must be positive")
    p = torch.arange(dim // 2, dtype=torch.float64)
    amp = 1.0
    if scaling is None:
        f = theta ** (-2.0 * p / dim)
    else:
        kind, s = scaling[0], float(scaling[1]) if len(scaling) > 1 else 0.0
        if not s > 0 or not math.isfinite(s):
            raise ValueError("the scaling factor must be positive")
        if kind == "linear" and len(scaling) == 2:
            f = theta ** (-2.0 * p / dim) / s
        elif kind == "ntk" and len(scaling) == 2:
            f = (theta * s ** (dim / (dim - 2)) if dim > 2 else theta) ** (-2.0 * p / dim)
        elif kind == "yarn" and len(scaling) in (3, 5):
            fast, slow = (32.0, 1.0) if len(scaling) == 3 else scaling[3:]
            if not fast > slow or not scaling[2] > 0:
                raise ValueError("yarn needs a positive context and fast > slow")
            f = theta ** (-2.0 * p / dim)
            keep = ((scaling[2] * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
            f = f * keep + f / s * (1 - keep)
            amp = max(1.0, 0.1 * math.log(s) + 1.0)
        else:
            raise ValueError("scaling must be None, ('linear', s), ('ntk', s) or "
                             "('yarn', s, context[, fast, slow])")
    return f.to(device), amp


def _positions(positions, N, B, dev):
    if positions.dtype not in (torch.int64, torch.int32) or positions.get_device() != dev or \
            not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int32 or int64 tensor on cuda:%d" % dev)
    if positions.shape != (N,) and positions.shape != (B, N):
        raise ValueError("positions must be [N] or [B, N]")
    return positions.data_ptr(), int(positions.dtype is torch.int64), \
        (N if positions.dim() == 2 else 0)


def _freqs(inv_freq, dev):
    if inv_freq.dtype is not torch.float64 or inv_freq.get_device() != dev or \
            inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 vector on cuda:%d" % dev)
    return inv_freq.data_ptr(), 2 * inv_freq.numel()


def rope(x, positions, inv_freq, layout="interleaved", amplitude=1.0, inverse=False, out=None,
         stream=None):
    """sage_rope on x [B, H, N, D] (bf16, fp16 or fp32 CUDA, unit channel
    stride, any others).  positions: int32/int64 [N] or [B, N]; inv_freq: fp64
    [R / 2] (rope_freqs), R <= D channels are turned.  layout: "interleaved"
    pairs (2p, 2p + 1), "half" pairs (p, p + R/2).  inverse: turn back -- the
    gradient of the forward call with respect to x, from that of its result;
    autograd takes it so where x requires a gradient (positions and inv_freq
    have none, and out cannot be given).  out: None, a tensor like x, or x
    itself; one that shares memory with x in another way is written by a copy
    of the result."""
    kind = _type(x)
    if x.dim() != 4 or kind < 0:
        raise ValueError("x must be a bf16, fp16 or fp32 tensor [B, H, N, D]")
    if layout not in ("interleaved", "half"):
        raise ValueError("layout must be 'interleaved' or 'half'")
    st = _here(x, stream)
    if st is None:
        with _There(x, stream):
            return rope(x, positions, inv_freq, layout, amplitude, inverse, out)
    if (x.requires_grad or inv_freq.requires_grad) and torch.is_grad_enabled():
        if inv_freq.requires_grad:
            raise ValueError("inv_freq has no gradient: detach it")
        if out is not None:
            raise ValueError("out cannot be given where x requires a gradient")
        return _Turn.apply(x, positions, inv_freq, layout, amplitude, inverse)
    B, H, N, D = x.shape
    dev = x.get_device()
    pos, p64, pstride = _positions(positions, N, B, dev)
    freq, R = _freqs(inv_freq, dev)
    if R > D:
        raise ValueError("inv_freq has more pairs than the heads")
    xs = _strides(x)
    if out is None:
        out, ys = _new(x)
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
        raise ValueError("out must have x's shape, type and device")
    else:
        ys = _out_strides(out)
        if _meets(x, xs, out, ys):
            return out.copy_(rope(x, positions, inv_freq, layout, amplitude, inverse))
    if B and H and N and D:
        _check(_lib().sage_rope(x.data_ptr(), out.data_ptr(), kind, B, H, N, D, R, xs, ys, pos, p64,
                                pstride, freq, amplitude, layout == "half", bool(inverse), st),
               "sage_rope")
    return out


def rope_tables(positions, inv_freq, amplitude=1.0, stream=None):
    """sage_rope_tables: (cos, sin), f32 [N, R / 2], the tables quant_qk and
    quant_qk_window take (R = D, interleaved pairs)."""
    st = _here(positions, stream)
    if st is None:
        with _There(positions, stream):
            return rope_tables(positions, inv_freq, amplitude)
    dev = positions.get_device()
    if positions.dim() != 1:
        raise ValueError("positions must be [N]")
    N = positions.shape[0]
    pos, p64, _ = _positions(positions, N, 1, dev)
    freq, R = _freqs(inv_freq, dev)
    c = torch.empty((N, R // 2), dtype=torch.float32, device=positions.device)
    s = torch.empty_like(c)
    if c.numel():
        _check(_lib().sage_rope_tables(N, R, pos, p64, freq, amplitude, c.data_ptr(), s.data_ptr(),
                                       st), "sage_rope_tables")
    return c, s


# ---------------------------------------------------------------- cache

class KVCache8:
    """Pages of an 8-bit key/value cache: k_i8 int8 [P, heads, 64, D], k_scale
    f32 [P, heads], v_f8 uint8 (e4m3 codes) like k_i8, v_exp int8 [P, heads]
    and, with track_weight, weight f32 [P, heads, 64]."""

    def __init__(self, num_pages, kv_heads, head_dim, device="cuda", track_weight=False):
        import torch
        shape = (int(num_pages), int(kv_heads), PAGE, int(head_dim))
        self._bind(torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape[:2], dtype=torch.float32, device=device),
                   torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.full(shape[:2], MIN_V_EXP, dtype=torch.int8, device=device),
                   torch.zeros(shape[:3], dtype=torch.float32, device=device)
                   if track_weight else None)

    @classmethod
    def from_buffers(cls, k_i8, k_scale, v_f8, v_exp, weight=None):
        """A cache over existing CUDA tensors of the layouts above."""
        self = cls.__new__(cls)
        self._bind(k_i8, k_scale, v_f8, v_exp, weight)
        return self

    def _bind(self, k_i8, k_scale, v_f8, v_exp, weight):
        import torch
        if k_i8.dim() != 4 or k_i8.shape[2] != PAGE or k_i8.shape[3] not in (64, 128):
            raise ValueError("codes must be [pages, heads, %d, 64 or 128]" % PAGE)
        P, h, _, D = k_i8.shape
        for t, shape, dt, what in ((k_i8, (P, h, PAGE, D), torch.int8, "k_i8"),
                                   (k_scale, (P, h), torch.float32, "k_scale"),
                                   (v_f8, (P, h, PAGE, D), torch.uint8, "v_f8"),
                                   (v_exp, (P, h), torch.int8, "v_exp"),
                                   (weight, (P, h, PAGE), torch.float32, "weight")):
            if t is None and what == "weight":
                continue
            if tuple(t.shape) != shape or t.dtype != dt or not t.is_contiguous() or \
                    not t.is_cuda or t.device != k_i8.device:
                raise ValueError("%s must be a contiguous %s CUDA tensor %s on one device"
                                 % (what, dt, shape))
        self.k_i8, self.k_scale, self.v_f8, self.v_exp, self.weight = (k_i8, k_scale, v_f8, v_exp,
                                                                        weight)
        self.num_pages, self.kv_heads, self.head_dim = P, h, D
        self.device, self.index = k_i8.device, k_i8.get_device()

    def struct(self, weight=None):
        w = self.weight if weight is None else weight
        return _Cache(self.k_i8.data_ptr(), self.k_scale.data_ptr(), self.v_f8.data_ptr(),
                      self.v_exp.data_ptr(), None if w is None else w.data_ptr(), self.num_pages,
                      self.kv_heads, self.head_dim)


def _seqs(cache, pages, lengths):
    if pages.dim() != 2:
        raise ValueError("pages must be [B, max_pages]")
    B, width = pages.shape
    return _Seqs(_int32(pages, (B, width), "pages", cache.index),
                 _int32(lengths, (B,), "lengths", cache.index), B, width)


def cache_append(cache, k, v, pages, lengths, n_new=None, k_shift=None, stream=None):
    """sage_cache_append: k, v [B, heads, n, D] (bf16 or fp16, unit channel
    stride) behind the `lengths` tokens that the sequences hold; the caller
    advances lengths.  n_new: int32 [B], tokens of each sequence (None: n).
    k_shift: f32 [heads, D] subtracted from the keys, or None."""
    st = _here(cache.k_i8, stream)
    if st is None:
        with _There(cache.k_i8, stream):
            return cache_append(cache, k, v, pages, lengths, n_new, k_shift)
    sq = _seqs(cache, pages, lengths)
    shape = k.shape
    if len(shape) != 4 or shape[0] != sq.B or shape[1] != cache.kv_heads or \
            shape[3] != cache.head_dim or v.shape != shape:
        raise ValueError("k and v must be [B, %d, n, %d]" % (cache.kv_heads, cache.head_dim))
    kind = _type(k)
    if kind not in (0, 1) or v.dtype is not k.dtype or k.get_device() != cache.index or \
            v.get_device() != cache.index:
        raise ValueError("k and v must be bf16 or fp16 tensors on %s" % cache.device)
    _shift_ok(cache, k_shift)
    nn = None if n_new is None else _int32(n_new, (sq.B,), "n_new", cache.index)
    if shape[2] == 0 or sq.B == 0:
        return
    _check(_lib().sage_cache_append(
        ctypes.byref(cache.struct()), ctypes.byref(sq), k.data_ptr(), v.data_ptr(), kind,
        shape[2], _strides(k), _strides(v), nn,
        None if k_shift is None else k_shift.data_ptr(), st), "sage_cache_append")


def _shift_ok(cache, k_shift):
    if k_shift is not None and (tuple(k_shift.shape) != (cache.kv_heads, cache.head_dim) or
                                k_shift.dtype != torch.float32 or not k_shift.is_contiguous() or
                                k_shift.device != cache.device):
        raise ValueError("k_shift must be a contiguous float32 tensor [%d, %d] on %s" % (
            cache.kv_heads, cache.head_dim, cache.device))


def cache_read(cache, pages, lengths, n, starts=None, k_shift=None, weights=False, stream=None):
    """sage_cache_read: (k, v), f32 [B, heads, n, D], of n tokens of each
    sequence from token starts[b] (int32 [B]; None: 0) on, zero where there is
    none; with `weights` also their summed weights, f32 [B, heads, n]."""
    st = _here(cache.k_i8, stream)
    if st is None:
        with _There(cache.k_i8, stream):
            return cache_read(cache, pages, lengths, n, starts, k_shift, weights)
    sq = _seqs(cache, pages, lengths)
    _shift_ok(cache, k_shift)
    sp = None if starts is None else _int32(starts, (sq.B,), "starts", cache.index)
    if weights and cache.weight is None:
        raise ValueError("the cache keeps no weights")
    k = cache.k_scale.new_empty((sq.B, cache.kv_heads, n, cache.head_dim))
    v = torch.empty_like(k)
    w = k.new_empty(k.shape[:3]) if weights else None
    if k.numel():
        _check(_lib().sage_cache_read(
            ctypes.byref(cache.struct()), ctypes.byref(sq), n, sp,
            None if k_shift is None else k_shift.data_ptr(), k.data_ptr(), v.data_ptr(),
            None if w is None else w.data_ptr(), st), "sage_cache_read")
    return (k, v, w) if weights else (k, v)


def _mask(mask):
    if mask is None or mask == "none":
        return 0, 0, 0, 0
    if mask == "causal":
        return 1, 0, 0, 0
    if isinstance(mask, tuple) and mask and mask[0] == "block_causal" and len(mask) == 2:
        return 2, int(mask[1]), 0, 0
    if isinstance(mask, tuple) and mask and mask[0] == "window" and len(mask) == 4:
        return 3, int(mask[1]), int(mask[2]), int(mask[3])
    raise ValueError(_MASKS)


def _query(q, cache, sq, q_lens, max_len, scale):
    kind = _type(q)
    if q.dim() != 4 or kind not in (0, 1) or q.get_device() != cache.index:
        raise ValueError("q must be a bf16 or fp16 tensor [B, H, Nq, D] on %s" % cache.device)
    B, H, N, D = q.shape
    if B != sq.B or D != cache.head_dim or H % cache.kv_heads:
        raise ValueError("q must be [B, H, Nq, %d], H a multiple of %d" % (cache.head_dim,
                                                                         cache.kv_heads))
    cap = sq.max_pages * PAGE
    return _Query(q.data_ptr(), _strides(q),
                  None if q_lens is None else _int32(q_lens, (B,), "q_lens", cache.index),
                  kind, H, N, cap if max_len is None or max_len > cap else max_len,
                  D ** -0.5 if scale is None else scale)


@functools.lru_cache(maxsize=256)
def _attn_workspace(dev, *shape):
    """sage_cache_attn_workspace_bytes of the current device, which is dev."""
    return _L.sage_cache_attn_workspace_bytes(*shape)


def cache_attn_workspace_bytes(cache, B, H, Nq, max_len, mask=None):
    """sage_cache_attn_workspace_bytes on the cache's device."""
    with _There(cache.k_i8, None):
        n = _lib().sage_cache_attn_workspace_bytes(B, cache.kv_heads, H, Nq, cache.head_dim,
                                                   int(max_len), *_mask(mask))
    if n == 0:
        raise ValueError("invalid shape or mask")
    return int(n)


def cache_attn(q, cache, pages, lengths, mask=None, q_lens=None, max_len=None, scale=None,
               out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """sage_cache_attn: attention of q [B, H, Nq, D] (bf16 or fp16, unit
    channel stride) over the cached tokens; returns out, or (out, lse).

    mask: None, "causal", ("block_causal", n) or ("window", frame_len,
    window_frames, sink_tokens).  q_lens: int32 [B], query rows of each
    sequence (None: Nq); other rows of out are left as they are.  max_len: a
    bound on the lengths known to the host (None: what the page table holds);
    it only chooses how the work is cut.  scale: None is 1 / sqrt(D).  out:
    None, a tensor like q, or q itself; one that shares memory with q in
    another way is written by a copy of the result."""
    st = _here(cache.k_i8, stream)
    if st is None:
        with _There(cache.k_i8, stream):
            return cache_attn(q, cache, pages, lengths, mask, q_lens, max_len, scale, out, lse,
                              return_lse, workspace)
    sq = _seqs(cache, pages, lengths)
    qs = _query(q, cache, sq, q_lens, max_len, scale)
    m = _mask(mask)
    if out is None:
        out, os = _new(q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != q.device:
        raise ValueError("out must have q's shape, type and device")
    else:
        os = _out_strides(out)
        if _meets(q, qs.q_strides, out, os):
            r = cache_attn(q, cache, pages, lengths, mask, q_lens, max_len, scale, torch.clone(out),
                           lse, return_lse, workspace)
            out.copy_(r[0] if return_lse else r)
            return (out, r[1]) if return_lse else out
    if lse is None:
        if return_lse:
            lse = cache.k_scale.new_empty(q.shape[:3])
    elif lse.shape != q.shape[:3] or lse.dtype != torch.float32 or lse.device != q.device or \
            not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [B, H, Nq]")
    if sq.B == 0 or qs.H == 0 or qs.Nq == 0:
        return (out, lse) if return_lse else out
    L = _lib()
    if workspace is None:
        n = _attn_workspace(cache.index, sq.B, cache.kv_heads, qs.H, qs.Nq, cache.head_dim,
                            qs.max_len, *m)
        if n > 16:  # else: one range a query tile, no partial results
            workspace = q.new_empty((n,), dtype=torch.uint8)
    elif workspace.device != q.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % q.device)
    ws, nb = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                  workspace.numel() * workspace.element_size())
    _check(L.sage_cache_attn(ctypes.byref(cache.struct()), ctypes.byref(sq), ctypes.byref(qs), *m,
                             out.data_ptr(), os, None if lse is None else lse.data_ptr(), ws, nb,
                             st), "sage_cache_attn")
    return (out, lse) if return_lse else out


def cache_weights(q, cache, lse, pages, lengths, mask=None, q_lens=None, max_len=None, scale=None,
                  weight=None, accumulate=True, stream=None):
    """sage_cache_weights: the attention weight that each cached token got from
    the rows of q, from cache_attn's lse of the same arguments, added to (or,
    accumulate=False, written over) cache.weight -- or `weight`, a float32
    tensor [pages, heads, 64].  Returns that tensor."""
    st = _here(cache.k_i8, stream)
    if st is None:
        with _There(cache.k_i8, stream):
            return cache_weights(q, cache, lse, pages, lengths, mask, q_lens, max_len, scale, weight,
                                 accumulate)
    sq = _seqs(cache, pages, lengths)
    qs = _query(q, cache, sq, q_lens, max_len, scale)
    if lse.shape != q.shape[:3] or lse.dtype != torch.float32 or lse.device != q.device or \
            not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [B, H, Nq]")
    w = cache.weight if weight is None else weight
    if w is None:
        raise ValueError("the cache keeps no weights")
    if tuple(w.shape) != tuple(cache.k_i8.shape[:3]) or w.dtype != torch.float32 or \
            w.device != cache.device or not w.is_contiguous():
        raise ValueError("weight must be a contiguous float32 tensor [pages, heads, %d]" % PAGE)
    if sq.B == 0:
        return w
    _check(_lib().sage_cache_weights(
        ctypes.byref(cache.struct(w)), ctypes.byref(sq), ctypes.byref(qs), *_mask(mask),
        lse.data_ptr(), bool(accumulate), st), "sage_cache_weights")
    return w


def cache_evict(cache, pages, lengths, keep, sink=0, recent=0, pages_out=None, workspace=None,
                stream=None):
    """sage_cache_evict: cut every sequence and head to at most `keep` tokens,
    by cache.weight.  Returns (kept, lengths): int32 [B, heads, keep], the
    survivors' old places in order, then -1; int32 [B].  pages_out: int32 [B,
    >= ceil(keep / 64)], pages the survivors go to (none of them in `pages`);
    None: the sequences' own first pages."""
    st = _here(cache.k_i8, stream)
    if st is None:
        with _There(cache.k_i8, stream):
            return cache_evict(cache, pages, lengths, keep, sink, recent, pages_out, workspace)
    sq = _seqs(cache, pages, lengths)
    keep, sink, recent = int(keep), int(sink), int(recent)
    if cache.weight is None:
        raise ValueError("the cache keeps no weights")
    if keep < 1 or sink < 0 or recent < 0 or sink + recent > keep:
        raise ValueError("keep must be at least 1 and at least sink + recent")
    po, width = None, 0
    if pages_out is not None:
        if pages_out.dim() != 2 or pages_out.shape[1] * PAGE < keep:
            raise ValueError("pages_out must be [B, at least %d]" % -(-keep // PAGE))
        width = pages_out.shape[1]
        po = _int32(pages_out, (sq.B, width), "pages_out", cache.index)
    kept = lengths.new_empty((sq.B, cache.kv_heads, keep))
    out = torch.empty_like(lengths)
    if sq.B == 0:
        return kept, out
    if workspace is None:
        n = _lib().sage_cache_evict_workspace_bytes(sq.B, cache.kv_heads, cache.head_dim, keep,
                                                    po is None)
        workspace = lengths.new_empty((max(n, 16),), dtype=torch.uint8)
    elif workspace.device != cache.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % cache.device)
    _check(_lib().sage_cache_evict(
        ctypes.byref(cache.struct()), ctypes.byref(sq), keep, sink, recent, po, width,
        kept.data_ptr(), out.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), st), "sage_cache_evict")
    return kept, out
