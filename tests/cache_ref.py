"""Plain implementations, in 64 bits on the CPU, of the rotary positions and
the paged 8-bit cache, written from the operators' definitions: the reference
that the GPU tests compare with."""
import math

import numpy as np
import torch

PAGE, MIN_EXP = 64, -40


def e4m3_round(x):
    """fp64 values to the nearest e4m3 value, ties to the even code."""
    x = np.asarray(x, np.float64)
    _, ex = np.frexp(x)
    step = np.exp2(np.maximum(ex - 1, -6) - 3.0)
    return np.clip(np.round(x / step) * step, -448, 448)


def e4m3_decode(codes):
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m, s = (c >> 3) & 15, c & 7, np.where(c & 128, -1.0, 1.0)
    return s * np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))


def value_exp(a):
    e = MIN_EXP
    while 448.0 * 2.0 ** e < a:
        e += 1
    return e


class Cache:
    """Codes and scales as the library holds them, in numpy."""

    def __init__(self, kv):
        self.k = kv.k_i8.cpu().numpy().copy()
        self.s = kv.k_scale.cpu().numpy().copy()
        self.v = e4m3_decode(kv.v_f8.cpu().numpy())  # code values
        self.e = kv.v_exp.cpu().numpy().astype(np.int64)
        self.w = None if kv.weight is None else kv.weight.cpu().numpy().copy()

    def append(self, k, v, pages, before, n_new, shift=None):
        k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
        if shift is not None:
            k = (k - shift.double().cpu().numpy()[None, :, None]).astype(np.float32).astype(np.float64)
        for b in range(k.shape[0]):
            done = 0
            while done < n_new[b]:
                pos = before[b] + done
                blk, slot = divmod(pos, PAGE)
                m = min(PAGE - slot, n_new[b] - done)
                pg = pages[b][blk]
                for h in range(k.shape[1]):
                    nk, nv = k[b, h, done:done + m], v[b, h, done:done + m]
                    s = np.float32(np.abs(nk).max() / 127.0)
                    e = value_exp(np.abs(nv).max())
                    if slot:
                        s, e = max(s, self.s[pg, h]), max(e, self.e[pg, h])
                        old = self.k[pg, h, :slot].astype(np.float64) * float(self.s[pg, h])
                        self.k[pg, h, :slot] = np.round(old / float(s)) if s > 0 else 0
                        self.v[pg, h, :slot] = e4m3_round(
                            self.v[pg, h, :slot] * 2.0 ** float(self.e[pg, h] - e))
                    else:
                        self.k[pg, h] = 0
                        self.v[pg, h] = 0
                        if self.w is not None:
                            self.w[pg, h] = 0
                    self.k[pg, h, slot:slot + m] = np.clip(np.round(nk / float(s)), -127, 127) \
                        if s > 0 else 0
                    self.v[pg, h, slot:slot + m] = e4m3_round(nv * 2.0 ** float(-e))
                    self.s[pg, h], self.e[pg, h] = s, e
                    if self.w is not None:
                        self.w[pg, h, slot:slot + m] = 0
                done += m

    def same(self, kv):
        assert np.array_equal(self.k, kv.k_i8.cpu().numpy()), "key codes differ"
        assert np.array_equal(self.s, kv.k_scale.cpu().numpy()), "key scales differ"
        assert np.array_equal(self.e, kv.v_exp.cpu().numpy()), "value exponents differ"
        assert np.array_equal(self.v, e4m3_decode(kv.v_f8.cpu().numpy())), "value codes differ"
        if self.w is not None:
            assert np.array_equal(self.w, kv.weight.cpu().numpy()), "weights differ"

    def tokens(self, pages, length, h):
        """(K, V) of one sequence and head, fp64 [length, D]."""
        t = np.arange(length)
        pg = np.asarray(pages, np.int64)[t // PAGE]
        K = self.k[pg, h, t % PAGE].astype(np.float64) * self.s[pg, h][:, None].astype(np.float64)
        V = self.v[pg, h, t % PAGE] * np.exp2(self.e[pg, h].astype(np.float64))[:, None]
        return K, V

    def evict(self, pages, length, keep, sink, recent, h):
        """(kept, k codes, scales, v code values, exps, weights) of one head."""
        t = np.arange(length)
        pg = np.asarray(pages, np.int64)[t // PAGE]
        w = self.w[pg, h, t % PAGE].astype(np.float64)
        n = min(keep, length)
        if n == length:
            kept = t
        else:
            order = sorted(range(sink, length - recent),
                           key=lambda i: (-(math.inf if math.isnan(w[i]) else w[i]), i))
            kept = np.array(sorted(list(range(sink)) + order[:keep - sink - recent] +
                                   list(range(length - recent, length))))
        kc = self.k[pg, h, t % PAGE].astype(np.float64)[kept]
        ks = self.s[pg, h][kept]
        vv = (self.v[pg, h, t % PAGE] * np.exp2(self.e[pg, h].astype(np.float64))[:, None])[kept]
        nb = -(-n // PAGE)
        K, V = np.zeros((nb * PAGE, kc.shape[1])), np.zeros((nb * PAGE, kc.shape[1]))
        S, E = np.zeros(nb, np.float32), np.zeros(nb, np.int64)
        W = np.zeros(nb * PAGE, np.float32)
        W[:n] = self.w[pg, h, t % PAGE][kept]
        for i in range(nb):
            a, z = i * PAGE, min(n, (i + 1) * PAGE)
            tok = ks[a:z] * (np.abs(kc[a:z]).max(1).astype(np.float32) / np.float32(127))
            S[i], E[i] = tok.max(), value_exp(np.abs(vv[a:z]).max())
            if S[i] > 0:
                K[a:z] = np.clip(np.round(kc[a:z] * ks[a:z, None].astype(np.float64) / float(S[i])),
                                 -127, 127)
            V[a:z] = e4m3_round(vv[a:z] * 2.0 ** float(-E[i]))
        return kept, K.reshape(nb, PAGE, -1), S, V.reshape(nb, PAGE, -1), E, W.reshape(nb, PAGE)


def visible(mask, n, length):
    """[n, length]: which keys the last n tokens of `length` see."""
    see = np.zeros((n, length), bool)
    for i in range(n):
        g = i + length - n
        for j in range(length):
            if mask is None:
                ok = True
            elif g < 0:
                ok = False
            elif mask == "causal":
                ok = j <= g
            elif mask[0] == "block_causal":
                ok = j // mask[1] <= g // mask[1]
            else:
                _, frame, win, sink = mask
                if j < sink:
                    ok = True
                elif g < sink:
                    ok = False
                else:
                    d = (g - sink) // frame - (j - sink) // frame
                    ok = 0 <= d < win
            see[i, j] = ok
    return see


def attention(ref, q, pages, lengths, q_lens, mask, scale, lse_in=None):
    """fp64 (O, lse, sum of p |v|, score error scale) over a Cache, rows of
    sequences shorter than Nq as NaN; with lse_in the summed weights too."""
    q = q.double().cpu().numpy()
    B, H, N, D = q.shape
    Hkv = ref.k.shape[1]
    O = np.full((B, H, N, D), np.nan)
    L = np.full((B, H, N), np.nan)
    A = np.full((B, H, N, D), np.nan)
    E = np.zeros((B, H, N))
    W = np.zeros(ref.k.shape[:3]) if lse_in is not None else None
    for b in range(B):
        n, length = q_lens[b], lengths[b]
        see = visible(mask, n, length)
        for h in range(H):
            K, V = ref.tokens(pages[b], length, h // (H // Hkv))
            x = q[b, h, :n] @ K.T * scale
            mag = np.abs(q[b, h, :n]) @ np.abs(K.T) * scale
            E[b, h, :n] = np.where(see, mag, 0).max(1, initial=0)
            x = np.where(see, x, -np.inf)
            m = x.max(1, initial=-np.inf)
            p = np.exp(x - np.where(np.isinf(m), 0, m)[:, None])
            z = p.sum(1)
            O[b, h, :n] = p @ V / np.where(z > 0, z, 1)[:, None]
            A[b, h, :n] = p @ np.abs(V) / np.where(z > 0, z, 1)[:, None]
            with np.errstate(divide="ignore"):
                L[b, h, :n] = np.log(z) + m if length else -np.inf
            if W is not None:
                g = lse_in[b, h, :n]
                w = np.where(see, np.exp(x - np.where(np.isinf(g), 0, g)[:, None]), 0).sum(0)
                t = np.arange(length)
                np.add.at(W, (np.asarray(pages[b])[t // PAGE], h // (H // Hkv), t % PAGE), w)
    return O, L, A, E, W


def rope(x, positions, inv_freq, layout, amplitude, inverse):
    """fp64 [B, H, N, D]; positions [B, N] ints (exact), inv_freq fp64."""
    x = x.double().cpu().numpy().copy()
    R = 2 * len(inv_freq)
    ang = np.asarray(positions, np.float64)[:, None, :, None] * np.asarray(inv_freq)
    c, s = np.cos(ang) * amplitude, np.sin(ang) * amplitude * (-1 if inverse else 1)
    i = slice(0, R // 2) if layout == "half" else slice(0, R, 2)
    j = slice(R // 2, R) if layout == "half" else slice(1, R, 2)
    a, b = x[..., i].copy(), x[..., j].copy()
    x[..., i], x[..., j] = a * c - b * s, a * s + b * c
    return x


def make_pages(lengths, rng, spare=0, width=None):
    """Shuffled page tables (numpy int32 [B, width]) and the page count."""
    need = [-(-n // PAGE) for n in lengths]
    ids = rng.permutation(sum(need) + spare + 1)
    width = max([1] + need) if width is None else width
    tab, at = np.full((len(lengths), width), -7, np.int32), 0  # -7: never read
    for b, n in enumerate(need):
        tab[b, :n] = ids[at:at + n]
        at += n
    return tab, len(ids), ids[at:]


def half_step(x, dtype):
    """Half a step of `dtype` at |x| (its normal range)."""
    return np.abs(x) * (torch.finfo(dtype).eps / 2)
