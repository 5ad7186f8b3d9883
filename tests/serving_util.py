"""Random layers and caches for the serving operators, and their definitions in
64 bits (keys and values of every row materialised, one sequence at a time)."""
import numpy as np
import torch

import rank_joint_qkv_b200 as q

DEV = "cuda"
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# a value held as one 16-bit part and the rounding residual in a second one
PARTS = {"f32": 2.0 ** -24, "f16": 2.0 ** -22, "bf16": 2.0 ** -16}


def rows_as(x, cache, group=128):
    """Float rows [..., r] -> (stored rows, group scales or None, their values in float64)."""
    if cache in TORCH:
        s = x.to(TORCH[cache])
        return s, None, s.double()
    qmax = 7 if cache == "i4" else 127
    v = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    sc = (v.abs().amax(-1) / qmax).half()
    inv = torch.where(sc > 0, 1.0 / sc.float(), torch.zeros_like(sc, dtype=torch.float32))
    codes = (v * inv.unsqueeze(-1)).round().clamp(-qmax, qmax).to(torch.int8)
    values = (codes.double() * sc.double().unsqueeze(-1)).reshape(x.shape)
    codes = codes.reshape(x.shape)
    if cache == "i4":   # channel 2j in the low nibble
        codes = ((codes[..., 0::2] & 0xF) | ((codes[..., 1::2] & 0xF) << 4)).to(torch.uint8)
    return codes.contiguous(), sc.contiguous(), values


class Layer:
    """One layer's weights, a batch of caches of `lens` rows (room for `room` more) and a query latent."""

    def __init__(self, *, cache="f16", weight="f16", out="f32", H=4, d_h=64, r=256, lens=(5, 0, 130), room=7, group=128,
                 rope=False, kernel=q.QSVD_KERNEL_AUTO, seed=0, prefix=0, peak=2.0, out_proj=None, past=None,
                 max_len=None):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.B, self.H, self.d_h, self.r = len(lens), H, d_h, r
        self.E, self.lens, self.rope, self.weight = H * d_h, list(lens), rope, weight
        self.max_len = max_len or max(max(lens), 1) + room
        self.dims = q.make_dims(self.E, H, d_h, r, self.B, self.max_len, cache=cache, weight=weight, out=out, group=group,
                                rope=rope, kernel=kernel, out_proj=out_proj)
        rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        spectrum = (1.0 + torch.arange(r, device=DEV)).pow(-0.4)
        spectrum = spectrum * (r / spectrum.square().sum()).sqrt()
        up = lambda k: (rnd(r, self.E) * (k / r ** 0.5)).to(TORCH[weight])  # noqa: E731
        self.wuq, self.wuk, self.wuv = up(peak), up(1.0), up(1.0)
        self.wd = (rnd(self.E, r) / self.E ** 0.5).to(TORCH[weight])
        self.packed = q.qsvd_prepare_weights(self.dims, self.wd, self.wuq, self.wuk, self.wuv)
        self.cache, self.scales, self.values = rows_as(rnd(self.B, self.max_len, r) * spectrum, cache, group)
        if prefix:
            self.prefix, self.prefix_scales, self.prefix_values = rows_as(rnd(prefix, r) * spectrum, cache, group)
        else:
            self.prefix = self.prefix_scales = None
            self.prefix_values = torch.zeros(0, r, device=DEV, dtype=torch.float64)
        if past is not None and cache in TORCH:   # what rows behind a length hold has no bearing
            for b, n in enumerate(lens):
                self.cache[b, n:] = past
        self.qin = rnd(self.B, r) * spectrum
        self.lengths = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.out_dtype = TORCH[out]

    def empty_out(self):
        return torch.full((self.B, self.E), float("nan"), dtype=self.out_dtype, device=DEV)

    def exact(self, wo=None):
        """(output B x E, weights of the own rows B x max_len, bound on the error of a score in natural units).

        The bound: the query and the absorbed query each enter the tensor
        cores as two parts of the weight / cache type (relative error PARTS
        per element) and every sum of r or d_h terms is taken in float32, in
        an order of its own (error below its number of terms x 2^-24 of the
        sum of magnitudes); 2^-20 for the rotary table's float32 entries and
        the exponential."""
        f64 = torch.float64
        wq, wk, wv = (w.to(f64) for w in (self.wuq, self.wuk, self.wuv))
        H, d_h, tau = self.H, self.d_h, self.d_h ** -0.5
        out = torch.zeros(self.B, self.E, dtype=f64, device=DEV)
        self.spread = torch.zeros_like(out)   # sum_t p_t |v_t|, for the rounding of p
        w = torch.zeros(self.B, self.max_len, dtype=f64, device=DEV)
        u = max(PARTS[self.weight], PARTS["bf16"] if self.cache.dtype == torch.bfloat16 else 0.0) + \
            (self.r + self.d_h) * 2.0 ** -24
        P, worst = self.prefix_values.shape[0], 0.0
        for b, n in enumerate(self.lens):
            if n + P == 0:
                continue
            c = torch.cat([self.prefix_values, self.values[b, :n]])
            qb = (self.qin[b].to(f64) @ wq).view(H, d_h)
            k, v = (c @ wk).view(-1, H, d_h), (c @ wv).view(-1, H, d_h)
            ka = (c.abs() @ wk.abs()).view(-1, H, d_h)
            qa = (self.qin[b].to(f64).abs() @ wq.abs()).view(H, d_h)
            worst = max(worst, float(torch.einsum("thd,hd->th", ka, qa).max()) * tau * u)
            if self.rope:
                ang = torch.arange(P + n, device=DEV, dtype=f64)[:, None] * \
                    torch.pow(10000.0, -2.0 * torch.arange(d_h // 2, device=DEV, dtype=f64) / d_h)
                cos, sin = ang.cos()[:, None], ang.sin()[:, None]
                turn = lambda x, cs, sn: torch.cat([x[..., :d_h // 2] * cs - x[..., d_h // 2:] * sn,  # noqa: E731
                                                    x[..., d_h // 2:] * cs + x[..., :d_h // 2] * sn], -1)
                qb, k = turn(qb, cos[P + n - 1], sin[P + n - 1]), turn(k, cos, sin)
            p = torch.softmax(torch.einsum("thd,hd->th", k, qb) * tau, 0)
            out[b] = torch.einsum("th,thd->hd", p, v).reshape(-1)
            self.spread[b] = torch.einsum("th,thd->hd", p, v.abs()).reshape(-1)
            w[b, :n] = p[P:].sum(1)
        if wo is not None:
            out = out @ wo.to(f64)
        return out, w, worst + 2.0 ** -20


def close_weights(got, want, bound, lens):
    """Each weight within a relative 2 x 1.1 x bound (its score and the softmax's sum are each off by at most `bound`)
    and the float32 sum's rounding; rows behind the length are not looked at."""
    for b, n in enumerate(lens):
        g, w = got[b, :n].double(), want[b, :n]
        assert torch.isfinite(g).all()
        lim = (2.2 * bound + 64 * 2.0 ** -24) * w + 1e-30
        assert bool(((g - w).abs() <= lim).all()), (b, float(((g - w).abs() / lim).max()))


def rel_err(got, want):
    """max |got - want| / rms(want), the bar of the decode's outputs (2e-3 with 16-bit or quantised latents)."""
    want = want.double()
    rms = float(want.square().mean().sqrt())
    return float((got.double() - want).abs().max()) / max(rms, 1e-30)


def keep_rows(weights, n, budget, sink, recent):
    """The kept rows of one sequence, by the definition (numpy)."""
    if n <= budget:
        return list(range(n))
    key = [(float("-inf"), 1) if np.isnan(x) else (float(x) + 0.0, 0) for x in weights]
    mid = sorted(range(sink, n - recent), key=lambda t: (-key[t][0], key[t][1], t))[:budget - sink - recent]
    return sorted(list(range(sink)) + mid + list(range(n - recent, n)))
