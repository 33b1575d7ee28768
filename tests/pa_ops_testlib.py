"""Inputs and 64-bit references of the operators beside plain decode and prefill
(pa_decode_scores, pa_evict, pa_cross_attention, pa_decode_shared), in plain numpy."""
import numpy as np
import torch

EPS32 = 2.0 ** -24                      # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS32}


class Paged:
    """Sequences of the given lengths in blocks scattered over a pool, unwritten slots NaN.
    lead[s] = (group, tokens): the first tokens (whole blocks) are those of that group."""

    def __init__(self, lens, Hkv, B, D, dt, seed, lead=None, spare=3, scale_v=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.B, self.D, self.dt = [int(x) for x in lens], Hkv, B, D, dt
        lead = lead or [None] * len(lens)
        groups = {}
        for x in lead:
            if x is not None:
                groups[x[0]] = max(groups.get(x[0], 0), x[1])
        n_lead = {g: n // B for g, n in groups.items()}
        own = [-(-L // B) - (x[1] // B if x is not None else 0) for L, x in zip(self.lens, lead)]
        NB = sum(n_lead.values()) + sum(own) + spare
        perm = rng.permutation(NB)
        at = 0
        gb = {}
        for g, n in n_lead.items():
            gb[g] = perm[at:at + n]
            at += n
        self.width = max([1] + [-(-L // B) for L in self.lens])
        self.tables = np.full((len(lens), self.width), -1, np.int32)
        k = np.full((NB, Hkv, B, D), np.nan, np.float32)
        v = k.copy()
        drawn = lambda n: (rng.standard_normal((n, Hkv, B, D), dtype=np.float32),  # noqa: E731
                           scale_v * rng.standard_normal((n, Hkv, B, D), dtype=np.float32))
        for g in gb:
            k[gb[g]], v[gb[g]] = drawn(len(gb[g]))
        for s, L in enumerate(self.lens):
            nl = 0 if lead[s] is None else lead[s][1] // B
            if nl:
                self.tables[s, :nl] = gb[lead[s][0]][:nl]
            mine = perm[at:at + own[s]]
            at += own[s]
            self.tables[s, nl:nl + own[s]] = mine
            if own[s]:
                kk, vv = drawn(own[s])
                if L % B:
                    kk[-1, :, L % B:], vv[-1, :, L % B:] = np.nan, np.nan
                k[mine], v[mine] = kk, vv
        self.k, self.v = torch.from_numpy(k).to(dt), torch.from_numpy(v).to(dt)
        self.rng = rng

    def q(self, n, Hq):
        return torch.from_numpy(self.rng.standard_normal((n, Hq, self.D), dtype=np.float32)).to(self.dt)

    def rows(self, s, kvh, L=None):
        """K and V rows of the first L tokens, in 64 bits."""
        L = self.lens[s] if L is None else L
        i = np.arange(L)
        b, o = self.tables[s][i // self.B], i % self.B
        return (self.k[b, kvh, o].double().numpy().reshape(L, self.D), self.v[b, kvh, o].double().numpy().reshape(L, self.D))

    def cuda(self):
        return (self.k.cuda(), self.v.cuda(), torch.from_numpy(self.tables).cuda(),
                torch.tensor(self.lens, dtype=torch.int32).cuda())


def attend(q, k, v, scale):
    """One head, 64 bits: output rows, softmax weights, log-sum-exp (natural), and the sum of the
    magnitudes that each logit adds up (for error bounds)."""
    q = np.asarray(q, np.float64)
    if len(k) == 0:
        return np.zeros((len(q), v.shape[1])), np.zeros((len(q), 0)), np.full(len(q), -np.inf), np.zeros((len(q), 0))
    z = q @ k.T * scale
    m = z.max(1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(1, keepdims=True)
    return p / l @ v, p / l, (m + np.log(l))[:, 0], np.abs(q) @ np.abs(k).T * abs(scale)


def logit_error(mags, D):
    """Bound of a logit's error in natural units: exact products (or one rounding each in fp32),
    D additions of fp32, the scale's and the maximum's subtraction's roundings."""
    return (2 * D + 8) * EPS32 * mags


def output_tolerance(pr, v, out, mags, D):
    """Bound of an output row's error when the weights are rounded once to bf16: that rounding (2^-8 of each
    weight), the output's own, and the logits' errors in weights and sum."""
    h = HALF[torch.bfloat16]
    a = pr @ np.abs(v)
    return h * a + h * np.abs(out) + a * (4 * logit_error(mags, D).max(initial=0.0) + 64 * EPS32) + 1e-30
