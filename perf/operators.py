"""What is measured of the rotary positions and the 8-bit key/value cache.

Five operators, each in its plain form (elementary torch operations in 32
bits, 64 where 32 lose what matters) and as the library's call:

  rope     rotary positions of query or key heads
  append   new keys and values into the paged 8-bit cache
  attn     attention over the paged 8-bit cache
  weights  attention weight that every cached key received, summed over rows
  evict    the cache cut down to the keys of largest summed weight

The cache: pages of 64 tokens; for each page and head int8 key codes with one
fp32 scale (absmax / 127) and e4m3 value codes with one power-of-two exponent
(the smallest e with absmax <= 448 * 2^e, at least -40).
"""
import math

import torch

own = False

BLOCK = 64
MIN_EXP = -40
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token of 16 requests, their query heads
        dict(name="rope_token", op="rope", B=16, H=32, N=1, D=128, R=128, layout="half",
             scaling="none", dtype="bf16", far=30000, inverse=False),
        # a whole clip, channel pairs side by side, half of each head rotated,
        # frequencies scaled for a context eight times as long
        dict(name="rope_clip_scaled", op="rope", B=1, H=12, N=32760, D=128, R=64,
             layout="interleaved", scaling="yarn", dtype="bf16", far=262144, inverse=False),
        # a decode step: one token of each of 32 requests into its tail page
        dict(name="append_token", op="append", B=32, Hkv=8, n=1, before=4000, D=128,
             dtype="bf16", shift=False),
        # a denoised latent frame enters the streaming cache; it starts inside
        # a page, and the keys' channel offsets are taken off
        dict(name="append_frame", op="append", B=1, Hkv=24, n=2040, before=24480, D=128,
             dtype="bf16", shift=True),
        # one request, one token, a short cache: latency
        dict(name="attn_token_short", op="attn", B=1, Hkv=8, G=4, n=1, length=500, D=128,
             mask="causal", p1=0, p2=0, p3=0, dtype="bf16", ragged=False),
        # a decode batch of uneven lengths, grouped heads
        dict(name="attn_token_batch", op="attn", B=32, Hkv=8, G=4, n=1, length=16000, D=128,
             mask="causal", p1=0, p2=0, p3=0, dtype="bf16", ragged=True),
        # few requests with long caches, one head group for each key head
        dict(name="attn_token_long", op="attn", B=4, Hkv=8, G=8, n=1, length=131071, D=128,
             mask="causal", p1=0, p2=0, p3=0, dtype="fp16", ragged=False),
        # a latent frame against its streaming cache: frames of 2040 tokens,
        # every head with keys of its own
        dict(name="attn_frame", op="attn", B=1, Hkv=24, G=1, n=2040, length=26520, D=128,
             mask="block_causal", p1=2040, p2=0, p3=0, dtype="bf16", ragged=False),
        # weights that the newest tokens of two requests gave to their caches
        dict(name="weights_recent", op="weights", B=2, Hkv=8, G=4, n=32, length=32000, D=128,
             mask="causal", p1=0, p2=0, p3=0, dtype="bf16", ragged=True),
        # one token of a decode batch
        dict(name="weights_token", op="weights", B=16, Hkv=8, G=4, n=1, length=8000, D=128,
             mask="causal", p1=0, p2=0, p3=0, dtype="bf16", ragged=True),
        # a batch cut to a quarter of its keys
        dict(name="evict_batch", op="evict", B=8, Hkv=8, length=16000, keep=4096, sink=64,
             recent=512, D=128, ragged=True),
        # the streaming cache cut to four frames, its reference frame kept
        dict(name="evict_stream", op="evict", B=1, Hkv=24, length=26520, keep=8160, sink=2040,
             recent=2040, D=128, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "weights", "evict"])
    D = rng.choice([64, 128])
    if op == "rope":
        H, B = _log(rng, 1, 40), _log(rng, 1, 32)
        N = max(1, min(_log(rng, 1, 32760), 12 * 32760 * 128 // (B * H * D)))
        return dict(op=op, B=B, H=H, N=N, D=D, R=2 * rng.randint(1, D // 2),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    dtype=rng.choice(["bf16", "fp16"]), far=_log(rng, 100, 1000000),
                    inverse=rng.random() < 0.3)
    Hkv = _log(rng, 1, 24)
    if op == "append":
        n = _log(rng, 1, 2040)
        B = max(1, min(_log(rng, 1, 32), 24 * 2040 // (n * Hkv)))
        return dict(op=op, B=B, Hkv=Hkv, n=n, before=rng.choice([0, _log(rng, 1, 25000)]), D=D,
                    dtype=rng.choice(["bf16", "fp16"]), shift=rng.random() < 0.5)
    if op == "evict":
        length = _log(rng, 50, 26520)
        B = max(1, min(_log(rng, 1, 8), 24 * 26520 // (length * Hkv)))
        keep = max(1, int(length * rng.uniform(0.05, 0.33)))
        sink = rng.randint(0, keep // 3)
        return dict(op=op, B=B, Hkv=Hkv, length=length, keep=keep, sink=sink,
                    recent=rng.randint(0, keep // 3), D=D, ragged=rng.random() < 0.5)
    G = rng.choice([1, 2, 3, 4, 6, 7, 8])
    if op == "weights":
        n, length = _log(rng, 1, 64), _log(rng, 10, 32000)
        B = max(1, min(_log(rng, 1, 16), 2 * 8 * 32000 // (length * Hkv),
                       2 * 32 * 32 * 32000 // (Hkv * G * n * length)))
        n = max(1, min(n, 2 * 32 * 32 * 32000 // (B * Hkv * G * length)))
    else:
        n, length = (1, _log(rng, 1, 131071)) if rng.random() < 0.5 else (
            _log(rng, 2, 2040), _log(rng, 10, 26520))
        B = max(1, min(_log(rng, 1, 32), 4 * 8 * 131071 // (length * Hkv)))
        n = max(1, min(n, 24 * 2040 * 26520 // (B * Hkv * G * length)))
    mask = rng.choice(["none", "causal", "block_causal", "window"])
    p1 = {"none": 0, "causal": 0}.get(mask, _log(rng, 1, 2040))
    return dict(op=op, B=B, Hkv=Hkv, G=G, n=n, length=length, D=D, mask=mask, p1=p1,
                p2=rng.randint(1, 6) if mask == "window" else 0,
                p3=rng.randint(0, 500) if mask == "window" else 0,
                dtype=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.5)


# ------------------------------------------------------------------ the inputs

def _freqs(case):
    """Angle per position of each channel pair (fp64) and the amplitude."""
    R, theta, factor, L0 = case["R"], 10000.0, 8.0, 32768
    p = torch.arange(R // 2, dtype=torch.float64)
    s = case["scaling"]
    if s == "ntk":
        theta = theta * factor ** (R / (R - 2)) if R > 2 else theta
    f = theta ** (-2.0 * p / R)
    if s == "linear":
        f = f / factor
    if s == "yarn":
        turns = L0 * f / (2 * math.pi)
        ramp = ((turns - 1.0) / 31.0).clamp(0, 1)
        return f * ramp + f / factor * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _lengths(case):
    """Cached tokens of each sequence: part of the case, like its sizes."""
    import random
    B, L = case["B"], case["length"]
    if not case["ragged"]:
        return [L] * B
    rng = random.Random(B * 1000003 + L)
    return [L] + [max(1, int(L * (0.2 + 0.8 * rng.random()))) for _ in range(B - 1)]


def _pages(lengths, spare, rng):
    """Page ids of each sequence, in no order, and the number of pages."""
    need = [-(-n // BLOCK) for n in lengths]
    ids = list(range(sum(need) + spare))
    rng.shuffle(ids)
    width = max(need)
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n] + [0] * (width - n))
        at += n
    return torch.tensor(table, dtype=torch.int32, device="cuda"), len(ids), ids[at:]


def _exps(a):
    """The smallest e with a <= 448 * 2^e, at least MIN_EXP (448 = 1.75 * 2^8)."""
    m, x = torch.frexp(a)  # a = m * 2^x, m in [0.5, 1)
    return torch.where(a > 0, x - 9 + (m > 0.875).int(), MIN_EXP).clamp(min=MIN_EXP)


def _p2(e):
    """2^e in fp32, exactly, -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _fp8(x):
    return x.to(torch.float8_e4m3fn)


def _make_cache(P, Hkv, D, gen):
    """Pages filled as a model's keys (channel offsets) and values would."""
    dev = "cuda"
    off = torch.randn((1, Hkv, 1, D), device=dev, generator=gen)
    k_i8 = torch.empty((P, Hkv, BLOCK, D), dtype=torch.int8, device=dev)
    v_f8 = torch.empty((P, Hkv, BLOCK, D), dtype=torch.float8_e4m3fn, device=dev)
    k_scale = torch.empty((P, Hkv), device=dev)
    v_exp = torch.empty((P, Hkv), dtype=torch.int8, device=dev)
    for a in range(0, P, 1024):
        b = min(P, a + 1024)
        k = torch.randn((b - a, Hkv, BLOCK, D), device=dev, generator=gen) + off
        v = torch.randn((b - a, Hkv, BLOCK, D), device=dev, generator=gen)
        s = (k.abs().amax((2, 3)).double() / 127).float()
        e = _exps(v.abs().amax((2, 3)))
        k_scale[a:b], v_exp[a:b] = s, e.to(torch.int8)
        k_i8[a:b] = torch.round(k / s[..., None, None]).clamp(-127, 127).to(torch.int8)
        v_f8[a:b] = _fp8(v * _p2(-e)[..., None, None])
    return dict(k_i8=k_i8, k_scale=k_scale, v_f8=v_f8.view(torch.uint8), v_exp=v_exp)


def _handle(st, D, Hkv):
    """The library's cache over the state's buffers."""
    import bit_quantized_attention_sage_b200 as sage
    c = st["cache"]
    st["kv"] = sage.KVCache8.from_buffers(c["k_i8"], c["k_scale"], c["v_f8"], c["v_exp"],
                                          c.get("weight"))


def _mask_arg(case):
    return {"none": None, "causal": "causal", "block_causal": ("block_causal", case["p1"]),
            "window": ("window", case["p1"], case["p2"], case["p3"])}[case["mask"]]


def prepare(case, seed):
    import random
    rng = random.Random("%d %s" % (seed, case["op"]))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dev, D = case["op"], "cuda", case["D"]

    def normal(*shape):
        return torch.randn(shape, device=dev, generator=gen).to(DT[case["dtype"]])

    st = dict(case=case)
    if op == "rope":
        f, amp = _freqs(case)
        st["x"] = normal(case["B"], case["H"], case["N"], D)
        first = [rng.randint(0, case["far"]) for _ in range(case["B"])]
        st["positions"] = (torch.tensor(first)[:, None] + torch.arange(case["N"])).to(dev)
        st["inv_freq"], st["amp"] = f.to(dev), amp
        return st
    Hkv, B = case["Hkv"], case["B"]
    if op == "append":
        # sequences of different lengths: part of the case, like its sizes
        before = [max(0, case["before"] - 37 * i % 101) for i in range(B)]
        n = case["n"]
        st["pages"], P, _ = _pages([x + n for x in before], 2, rng)
        st["before"] = torch.tensor(before, dtype=torch.int32, device=dev)
        st["after"] = st["before"] + n
        st["starts"] = st["before"] // BLOCK * BLOCK
        # tokens of the touched pages, from the first touched page's start on
        st["span"] = max(x + n - x // BLOCK * BLOCK for x in before)
        st["k"] = normal(B, Hkv, n, D) + 2 * normal(1, Hkv, 1, D)
        st["v"] = normal(B, Hkv, n, D)
        st["shift"] = None
        if case["shift"]:
            st["shift"] = st["k"].float().mean((0, 2)).contiguous()
        st["cache"] = _make_cache(P, Hkv, D, gen)
        # a call changes what the tail page held only through a scale that
        # grows, and a second call finds it grown: its results are the same
        if own:
            _handle(st, D, Hkv)
        return st
    lengths = _lengths(case)
    st["host_lengths"], st["max_len"] = lengths, max(lengths)
    st["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    spare = 0
    if op == "evict":
        spare = B * -(-case["keep"] // BLOCK)
    st["pages"], P, left = _pages(lengths, spare, rng)
    st["cache"] = _make_cache(P, Hkv, D, gen)
    if op == "evict":
        # summed weights of many steps: a heavy tail, and equal ones among them
        w = torch.rand((P, Hkv, BLOCK), device=dev, generator=gen).pow(-0.5) - 1
        st["cache"]["weight"] = torch.where(w < 0.05, 0.0, w)
        st["pages_out"] = torch.tensor(left, dtype=torch.int32, device=dev).view(B, -1)
    else:
        st["q"] = normal(B, Hkv * case["G"], case["n"], D)
        if op == "weights":
            st["weight"] = torch.zeros((P, Hkv, BLOCK), device=dev)
            st["lse"] = torch.empty(st["q"].shape[:3], device=dev)
            for b in range(B):
                t, vis, _ = _scores(st, b, torch.float32)
                st["lse"][b] = torch.where(vis, t, -math.inf).logsumexp(-1).view(
                    -1, case["n"])
    if own:
        _handle(st, D, Hkv)
    return st


# ------------------------------------------------------------------ plain forms

def _visible(case, n, length):
    """[n, length] truth values: which keys each new token sees."""
    j = torch.arange(length, device="cuda")[None, :]
    g = (torch.arange(n, device="cuda") + length - n)[:, None]
    m = case["mask"]
    if m == "none":
        return torch.ones((n, length), dtype=torch.bool, device="cuda")
    if m == "causal":
        return j <= g
    if m == "block_causal":
        return (g >= 0) & (j // case["p1"] <= g // case["p1"])
    frame, win, sink = case["p1"], case["p2"], case["p3"]
    f = (g - sink) // frame
    inside = (j >= sink) & ((j - sink) // frame <= f) & ((j - sink) // frame > f - win)
    return (g >= 0) & ((j < sink) | ((g >= sink) & inside))


def _scores(st, b, dtype):
    """Scaled scores [Hkv, G * n, length] of sequence b, the mask, the pages."""
    case, c = st["case"], st["cache"]
    length, D = st["host_lengths"][b], case["D"]
    ids = st["pages"][b, :-(-length // BLOCK)].long()
    k = c["k_i8"][ids].to(dtype) * c["k_scale"][ids].to(dtype)[..., None, None]
    k = k.transpose(0, 1).reshape(case["Hkv"], -1, D)[:, :length]
    q = st["q"][b].to(dtype).reshape(case["Hkv"], case["G"] * case["n"], D)
    t = (q @ k.transpose(1, 2)) * (1.0 / math.sqrt(D))
    vis = _visible(case, case["n"], length).repeat(case["G"], 1)
    return t, vis, ids


def _plain_rope(st):
    case, x = st["case"], st["x"].float()
    R = case["R"]
    ang = st["positions"].double()[..., None] * st["inv_freq"]
    c = (torch.cos(ang) * st["amp"]).float()[:, None]
    s = (torch.sin(ang) * st["amp"]).float()[:, None]
    if case["inverse"]:
        s = -s
    y = x.clone()
    a, b = (slice(0, R // 2), slice(R // 2, R)) if case["layout"] == "half" else (
        slice(0, R, 2), slice(1, R, 2))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y.to(st["x"].dtype)


def _plain_append(st):
    """Values of the touched pages, [B, Hkv, span, D]: zero past the end."""
    case, c = st["case"], st["cache"]
    B, Hkv, n, D = st["k"].shape
    nb = -(-(st["span"]) // BLOCK)
    k = st["k"].float()
    if st["shift"] is not None:
        k = k - st["shift"][None, :, None]
    v = st["v"].float()
    out_k = torch.zeros((B, Hkv, nb * BLOCK, D), device=k.device)
    out_v = torch.zeros_like(out_k)
    first = (st["before"] // BLOCK).long()
    off = (st["before"] % BLOCK).long()
    # new tokens at their places, and what the tail page held before them
    at = off[:, None] + torch.arange(n, device=k.device)
    seq = torch.arange(B, device=k.device)
    new_k, new_v = torch.zeros_like(out_k), torch.zeros_like(out_k)
    new_k[seq[:, None], :, at] = k.transpose(1, 2)
    new_v[seq[:, None], :, at] = v.transpose(1, 2)
    page = st["pages"][seq, first].long()
    held = (torch.arange(BLOCK, device=k.device)[None, :] < off[:, None])[:, None, :, None]
    old_s = torch.where((off > 0)[:, None], c["k_scale"][page], 0.0)
    old_e = torch.where((off > 0)[:, None], c["v_exp"][page].int(), MIN_EXP)
    old_k = torch.where(held, c["k_i8"][page].double(), 0.0)
    old_v = torch.where(held, c["v_f8"][page].view(torch.float8_e4m3fn).float(), 0.0)
    nk = new_k.view(B, Hkv, nb, BLOCK, D)
    nv = new_v.view(B, Hkv, nb, BLOCK, D)
    s = (nk.abs().amax((3, 4)).double() / 127).float()
    e = _exps(nv.abs().amax((3, 4)))
    s[:, :, 0] = torch.maximum(s[:, :, 0], old_s)
    e[:, :, 0] = torch.maximum(e[:, :, 0], old_e)
    sd = torch.where(s > 0, s, 1.0).double()[..., None, None]
    codes = torch.round(nk.double() / sd).clamp(-127, 127)
    vals = _fp8(nv * _p2(-e)[..., None, None]).float()
    kept = torch.round(old_k * old_s.double()[..., None, None] / sd[:, :, 0]).clamp(-127, 127)
    kept_v = _fp8(old_v * _p2(old_e - e[:, :, 0])[..., None, None]).float()
    codes[:, :, 0] = torch.where(held, kept, codes[:, :, 0])
    vals[:, :, 0] = torch.where(held, kept_v, vals[:, :, 0])
    out_k = (codes.float() * s[..., None, None]).view(B, Hkv, -1, D)[:, :, :st["span"]]
    out_v = (vals * _p2(e)[..., None, None]).view(B, Hkv, -1, D)[:, :, :st["span"]]
    return out_k, out_v


def _plain_attn(st):
    case, c = st["case"], st["cache"]
    out, lse = torch.empty_like(st["q"]), torch.empty(st["q"].shape[:3], device="cuda")
    for b in range(case["B"]):
        t, vis, ids = _scores(st, b, torch.float32)
        t = t.masked_fill(~vis, -math.inf)
        m = t.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        p = torch.exp(t - m)
        z = p.sum(-1, keepdim=True)
        v = c["v_f8"][ids].view(torch.float8_e4m3fn).float()
        v = v * _p2(c["v_exp"][ids])[..., None, None]
        v = v.transpose(0, 1).reshape(case["Hkv"], -1, case["D"])[:, :t.shape[-1]]
        o = (p @ v) / torch.where(z > 0, z, 1.0)
        out[b] = o.reshape(out[b].shape).to(out.dtype)
        lse[b] = (torch.log(z) + m).view(lse[b].shape)
    return out, lse


def _plain_weights(st):
    case = st["case"]
    out = torch.zeros_like(st["weight"])
    for b in range(case["B"]):
        t, vis, ids = _scores(st, b, torch.float32)
        lse = st["lse"][b].view(case["Hkv"], -1, 1)
        w = torch.where(vis, torch.exp(t - torch.where(lse > -math.inf, lse, 0.0)), 0.0).sum(1)
        pad = torch.zeros((case["Hkv"], len(ids) * BLOCK), device="cuda")
        pad[:, :t.shape[-1]] = w
        out[ids] = pad.view(case["Hkv"], -1, BLOCK).transpose(0, 1)
    return out


def _plain_evict(st):
    case, c = st["case"], st["cache"]
    B, Hkv, D, keep = case["B"], case["Hkv"], case["D"], case["keep"]
    nb = -(-keep // BLOCK)
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    ck = torch.zeros((B, Hkv, nb * BLOCK, D), dtype=torch.float64, device="cuda")
    cv = torch.zeros((B, Hkv, nb * BLOCK, D), device="cuda")
    sk = torch.zeros((B, Hkv, nb * BLOCK), device="cuda")
    ev = torch.full((B, Hkv, nb * BLOCK), MIN_EXP, dtype=torch.int32, device="cuda")
    ow = torch.zeros((B, Hkv, nb * BLOCK), device="cuda")
    for b in range(B):
        length = st["host_lengths"][b]
        ids = st["pages"][b, :-(-length // BLOCK)].long()
        w = c["weight"][ids].transpose(0, 1).reshape(Hkv, -1)[:, :length]
        rank = w.clone()
        n = min(keep, length)
        rank[:, :case["sink"]] = math.inf
        rank[:, max(0, length - case["recent"]):] = math.inf
        top = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :n]
        top = torch.sort(top, dim=1)[0]
        kept[b, :, :n] = top.int()
        page, slot, h = ids[top // BLOCK], top % BLOCK, torch.arange(Hkv, device="cuda")[:, None]
        ck[b, :, :n] = c["k_i8"][page, h, slot].double()
        cv[b, :, :n] = c["v_f8"][page, h, slot].view(torch.float8_e4m3fn).float()
        sk[b, :, :n], ev[b, :, :n] = c["k_scale"][page, h], c["v_exp"][page, h].int()
        ow[b, :, :n] = w.gather(1, top)
    # a page's new scale is its largest token's
    s = (sk * (ck.abs().amax(-1) / 127).float()).view(B, Hkv, nb, BLOCK).amax(-1)
    e = _exps((cv * _p2(ev)[..., None]).abs().amax(-1)).view(B, Hkv, nb, BLOCK).amax(-1)
    st_ = s.repeat_interleave(BLOCK, -1)
    et = e.repeat_interleave(BLOCK, -1)
    sd = torch.where(st_ > 0, st_, 1.0).double()[..., None]
    codes = torch.round(ck * sk.double()[..., None] / sd).clamp(-127, 127)
    vals = _fp8(cv * _p2(ev - et)[..., None]).float()
    n_out = st["lengths"].clamp(max=keep)
    k = (codes.float() * st_[..., None])[:, :, :keep]
    v = (vals * _p2(et)[..., None])[:, :, :keep]
    return kept, n_out, k, v, ow[:, :, :keep]


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn,
                "weights": _plain_weights, "evict": _plain_evict}[op](st)
    import bit_quantized_attention_sage_b200 as sage
    if op == "rope":
        return sage.rope(st["x"], st["positions"], st["inv_freq"], layout=case["layout"],
                         amplitude=st["amp"], inverse=case["inverse"])
    kv = st["kv"]
    if op == "append":
        sage.cache_append(kv, st["k"], st["v"], st["pages"], st["before"], k_shift=st["shift"])
        return sage.cache_read(kv, st["pages"], st["after"], st["span"], starts=st["starts"])
    if op == "attn":
        return sage.cache_attn(st["q"], kv, st["pages"], st["lengths"], mask=_mask_arg(case),
                               max_len=st["max_len"], return_lse=True)
    if op == "weights":
        return sage.cache_weights(st["q"], kv, st["lse"], st["pages"], st["lengths"],
                                  mask=_mask_arg(case), max_len=st["max_len"],
                                  weight=st["weight"], accumulate=False)
    kept, n_out = sage.cache_evict(kv, st["pages"], st["lengths"], case["keep"],
                                   sink=case["sink"], recent=case["recent"],
                                   pages_out=st["pages_out"])
    k, v, w = sage.cache_read(kv, st["pages_out"], n_out, case["keep"], weights=True)
    return kept, n_out, k, v, w


def work(case):
    op, D = case["op"], case["D"]
    if op == "rope":
        size = 4 if case["dtype"] == "fp32" else 2
        el = case["B"] * case["H"] * case["N"]
        return {"bytes": el * D * 2 * size + case["B"] * case["N"] * 8,
                "flops": el * case["R"] * 3}
    Hkv, B = case["Hkv"], case["B"]
    if op == "append":
        # 16-bit keys and values in, fp32 values of the touched pages out
        span = case["before"] % BLOCK + case["n"]
        el = B * Hkv * D
        return {"bytes": el * (case["n"] * 4 + span * 8), "flops": el * case["n"] * 6}
    lengths = _lengths(case)
    total = sum(lengths)
    if op == "evict":
        n = sum(min(x, case["keep"]) for x in lengths)
        # every weight, the kept codes in, their fp32 values and weights out
        return {"bytes": Hkv * (total * 4 + n * (2 * D + 8 * D + 4 + 4)),
                "flops": Hkv * (total * 4 + n * D * 6)}
    rows = case["n"] * case["G"]
    n = case["n"]
    pairs = sum(_pairs(case, L) for L in lengths)
    used = total
    if case["mask"] == "window":
        used = sum(min(L, case["p3"] + case["p2"] * case["p1"] + n) for L in lengths)
    if op == "weights":
        return {"bytes": Hkv * (used * D + total * 4 + B * rows * (2 * D + 4)),
                "flops": Hkv * case["G"] * pairs * (2 * D + 2)}
    return {"bytes": Hkv * (used * 2 * D + B * rows * (4 * D + 4)),
            "flops": Hkv * case["G"] * pairs * (4 * D + 4)}


def _pairs(case, L):
    """(new token, key) pairs that the mask leaves, of one sequence."""
    n, tot = case["n"], 0
    for i in range(n):
        g = i + L - n
        if case["mask"] == "none":
            tot += L
        elif g < 0:
            continue
        elif case["mask"] == "causal":
            tot += g + 1
        elif case["mask"] == "block_causal":
            tot += min(L, (g // case["p1"] + 1) * case["p1"])
        else:
            frame, win, sink = case["p1"], case["p2"], case["p3"]
            tot += min(sink, L)
            if g >= sink:
                f = (g - sink) // frame
                lo = sink + max(0, f - win + 1) * frame
                tot += min(L, sink + (f + 1) * frame) - lo
    return tot


# ------------------------------------------------------------------ definitions in 64 bits

def _e4m3(x):
    """x (fp64) to the nearest e4m3 value, ties to the even one, |x| <= 448."""
    _, ex = torch.frexp(x)
    step = torch.exp2((ex - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def _pow_for(a):
    """2^e, the smallest power with a <= 448 * 2^e and e >= MIN_EXP (fp64)."""
    e = torch.ceil(torch.log2(a.double() / 448.0)).clamp(min=MIN_EXP)
    e = torch.where(448.0 * torch.exp2(e - 1) >= a, e - 1, e)
    e = torch.where(448.0 * torch.exp2(e) < a, e + 1, e)
    return torch.exp2(e.clamp(min=MIN_EXP))


def _full(st, b, what):
    """Values of one sequence's cache in fp64, [Hkv, pages * 64, D]."""
    c = st["cache"]
    ids = st["pages"][b].long()
    if what == "k":
        x = c["k_i8"][ids].double().mul(c["k_scale"][ids].double()[..., None, None])
    else:
        x = c["v_f8"][ids].view(torch.float8_e4m3fn).double()
        x = x * torch.exp2(c["v_exp"][ids].double())[..., None, None]
    return x.transpose(0, 1).flatten(1, 2)


def _exact_rope(st):
    case = st["case"]
    x, R = st["x"].double(), case["R"]
    ang = torch.outer(st["positions"].flatten().double(), st["inv_freq"])
    ang = ang.view(case["B"], 1, case["N"], R // 2)
    turn = st["amp"] * torch.complex(torch.cos(ang), torch.sin(ang))
    if case["inverse"]:
        turn = turn.conj()
    rot = x[..., :R]
    if case["layout"] == "half":
        w = torch.complex(rot[..., :R // 2].contiguous(), rot[..., R // 2:].contiguous()) * turn
        rot = torch.cat([w.real, w.imag], -1)
    else:
        w = torch.view_as_complex(rot.unflatten(-1, (-1, 2)).contiguous()) * turn
        rot = torch.view_as_real(w).flatten(-2)
    return torch.cat([rot, x[..., R:]], -1)


def _exact_append(st):
    case, c = st["case"], st["cache"]
    B, Hkv, n, D = st["k"].shape
    out_k = torch.zeros((B, Hkv, st["span"], D), dtype=torch.float64, device="cuda")
    out_v = torch.zeros_like(out_k)
    before = st["before"].tolist()
    for b in range(B):
        k, v = st["k"][b].double(), st["v"][b].double()
        if st["shift"] is not None:
            k = (k - st["shift"].double()[:, None]).float().double()
        base, done = before[b] // BLOCK * BLOCK, 0
        while done < n:
            pos = before[b] + done
            slot, blk = pos % BLOCK, pos // BLOCK
            m = min(BLOCK - slot, n - done)
            nk, nv = k[:, done:done + m], v[:, done:done + m]
            s = (nk.abs().amax((1, 2)) / 127).float().double()
            p = _pow_for(nv.abs().amax((1, 2)))
            at = blk * BLOCK - base
            if slot:
                pg = int(st["pages"][b, blk])
                s0, p0 = c["k_scale"][pg].double(), torch.exp2(c["v_exp"][pg].double())
                s, p = torch.maximum(s, s0), torch.maximum(p, p0)
                ok = c["k_i8"][pg, :, :slot].double() * s0[:, None, None]
                ov = c["v_f8"][pg, :, :slot].view(torch.float8_e4m3fn).double() * p0[:, None, None]
                sp = torch.where(s > 0, s, 1.0)[:, None, None]
                out_k[b, :, at:at + slot] = torch.round(ok / sp).clamp(-127, 127) * s[:, None, None]
                out_v[b, :, at:at + slot] = _e4m3(ov / p[:, None, None]) * p[:, None, None]
            sp = torch.where(s > 0, s, 1.0)[:, None, None]
            out_k[b, :, at + slot:at + slot + m] = (
                torch.round(nk / sp).clamp(-127, 127) * s[:, None, None])
            out_v[b, :, at + slot:at + slot + m] = _e4m3(nv / p[:, None, None]) * p[:, None, None]
            done += m
    return out_k, out_v


def _exact_attn(st, weights=False):
    case = st["case"]
    n, G, D = case["n"], case["G"], case["D"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    w = torch.zeros(st["weight"].shape, dtype=torch.float64, device="cuda") if weights else None
    for b in range(case["B"]):
        L = st["host_lengths"][b]
        K = _full(st, b, "k")[:, :L]
        V = None if weights else _full(st, b, "v")[:, :L]
        see = _visible(case, n, L)
        for h in range(case["Hkv"] * G):
            x = st["q"][b, h].double() @ K[h // G].T / math.sqrt(D)
            x = x.masked_fill(~see, -math.inf)
            if weights:
                g = st["lse"][b, h].double()[:, None]
                col = torch.exp(x - torch.where(g > -math.inf, g, 0.0)).sum(0)
                w_pad = torch.zeros(-(-L // BLOCK) * BLOCK, dtype=torch.float64, device="cuda")
                w_pad[:L] = col
                w[st["pages"][b, :-(-L // BLOCK)].long(), h // G] += w_pad.view(-1, BLOCK)
            else:
                lse[b, h] = torch.logsumexp(x, -1)
                z = torch.where(lse[b, h] > -math.inf, lse[b, h], 0.0)
                out[b, h] = torch.exp(x - z[:, None]) @ V[h // G]
    return w if weights else (out, lse)


def _exact_evict(st):
    case, c = st["case"], st["cache"]
    B, Hkv, D, keep = case["B"], case["Hkv"], case["D"], case["keep"]
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32)
    k = torch.zeros((B, Hkv, keep, D), dtype=torch.float64, device="cuda")
    v = torch.zeros_like(k)
    wt = torch.zeros((B, Hkv, keep), dtype=torch.float64, device="cuda")
    W = c["weight"].double()
    for b in range(B):
        L = st["host_lengths"][b]
        n = min(L, keep)
        fullw = W[st["pages"][b].long()].transpose(0, 1).flatten(1)[:, :L]
        KC = c["k_i8"][st["pages"][b].long()].transpose(0, 1).flatten(1, 2).double()
        KS = c["k_scale"][st["pages"][b].long()].double().T.repeat_interleave(BLOCK, 1)
        V = _full(st, b, "v")
        forced = set(range(min(case["sink"], L))) | set(range(max(0, L - case["recent"]), L))
        for h in range(Hkv):
            if n == L:
                idx = list(range(L))
            else:
                wl = fullw[h].tolist()
                rest = sorted((i for i in range(L) if i not in forced), key=lambda i: (-wl[i], i))
                idx = sorted(list(forced) + rest[:n - len(forced)])
            kept[b, h, :n] = torch.tensor(idx, dtype=torch.int32)
            ix = torch.tensor(idx, device="cuda")
            wt[b, h, :n] = fullw[h, ix]
            kc, ks, vv = KC[h, ix], KS[h, ix], V[h, ix]
            part = (kc.abs().amax(1) / 127).float().double()
            tok = (ks * part).float().double()
            for i in range(0, n, BLOCK):
                j = min(n, i + BLOCK)
                s = tok[i:j].amax()
                p = _pow_for(vv[i:j].abs().amax())
                if s > 0:
                    k[b, h, i:j] = torch.round(kc[i:j] * ks[i:j, None] / s).clamp(-127, 127) * s
                v[b, h, i:j] = _e4m3(vv[i:j] / p) * p
    n_out = torch.tensor([min(x, keep) for x in st["host_lengths"]], dtype=torch.int32)
    return kept.cuda(), n_out.cuda(), k, v, wt


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn,
            "weights": lambda s: _exact_attn(s, True), "evict": _exact_evict}[case["op"]](st)
