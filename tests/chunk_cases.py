"""Inputs of the dense chunk attention's tests and its plain implementation (NumPy, 64 bits), with a
bound of the error that the kernel's documented roundings allow. Written from the definition; nothing
here uses the library."""
from __future__ import annotations

import numpy as np

from tests.step_cases import E4M3, GRID, blocks_of
from workloads.gen import bf16_from_f32, f32_from_bf16

E4M3_ALL = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
E2M1_ALL = np.concatenate([GRID, -GRID])
NVFP4, FP8 = 0, 1
ROW = {NVFP4: 352, FP8: 576}


def row_values(rows, fmt, latent_scale=1.0, rope_scale=1.0):
    """Latent [n, 512] and rope [n, 64] values of cache rows (uint8 [n, row bytes])."""
    rope = E4M3_ALL[rows[:, -64:]] * rope_scale
    if fmt == FP8:
        return E4M3_ALL[rows[:, :512]] * latent_scale, rope
    lat = np.empty((len(rows), 512))
    lat[:, 0::2], lat[:, 1::2] = E2M1_ALL[rows[:, :256] & 15], E2M1_ALL[rows[:, :256] >> 4]
    return lat * np.repeat(E4M3_ALL[rows[:, 256:288]], 16, 1), rope


def random_rows(rng, n, fmt):
    """Rows of values around 1: codes of all kinds, scales 2^-3 .. 2^1, rope values of E4M3 up to 3.75."""
    rows = rng.integers(0, 256, (n, ROW[fmt]), dtype=np.uint8)
    e4m3 = lambda shape, lo, hi: (rng.integers(lo, hi, shape) | (rng.integers(0, 2, shape) << 7)).astype(np.uint8)
    if fmt == NVFP4:
        rows[:, 256:288] = rng.integers(0x20, 0x40, (n, 32))
    else:
        rows[:, :512] = e4m3((n, 512), 0, 0x48)
    rows[:, -64:] = e4m3((n, 64), 0, 0x48)
    return rows


class Case:
    def __init__(self, seed, lens, new, heads, fmt=NVFP4, page=64, pad=0, stride_pad=0, spare=3, width=None,
                 latent_scale=1.0, rope_scale=1.0, sm_scale=1 / 24, q_scale=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
        self.H, self.fmt, self.page, self.sm_scale = heads, fmt, page, sm_scale
        self.latent_scale, self.rope_scale = latent_scale, rope_scale
        self.S = len(lens)
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.n = int(self.cu[-1])
        self.num_q = self.n + pad
        pages = [blocks_of(int(x), page) for x in lens]
        self.width = width or max(max(pages), 1)
        self.blocks = sum(pages) + spare
        self.stride = page * ROW[fmt] + stride_pad
        perm, at = rng.permutation(self.blocks).astype(np.int32), 0
        self.table = np.full((self.S, self.width), -1, np.int32)
        for s, k in enumerate(pages):
            self.table[s, :k] = perm[at:at + k]
            at += k
        self.pool = rng.integers(0, 256, (self.blocks, self.stride), dtype=np.uint8)
        self.pool[:, :page * ROW[fmt]] = random_rows(rng, self.blocks * page, fmt).reshape(self.blocks, -1)
        q = rng.standard_normal((max(self.num_q, 1), heads, 576))[:self.num_q] * q_scale
        self.ql, self.qr = bf16_from_f32(q[..., :512].astype(np.float32)), bf16_from_f32(q[..., 512:].astype(np.float32))

    def keys(self, s):
        """Latent, rope and existence of the positions of sequence s."""
        L = int(self.lens[s])
        pos = np.arange(L)
        pages = self.table[s, pos // self.page] if L else np.zeros(0, np.int32)
        ok = (pages >= 0) & (pages < self.blocks)
        rows = self.pool[:, :self.page * ROW[self.fmt]].reshape(self.blocks, self.page, -1)
        lat, rope = row_values(rows[np.where(ok, pages, 0), pos % self.page], self.fmt, self.latent_scale,
                               self.rope_scale)
        return lat, rope, ok

    def reference(self, tokens=None):
        """(out, lse, bound of |out error|, bound of |lse error|) of all tokens, or of some rows.

        The kernel's roundings: FP16 weights, off by 2^-11 of themselves (half a step) or, where
        subnormal, by half of their step of 2^-24; the largest weight is at least 2^2 then, so that
        relative to it that is 2^-25 / 2^2 = 2^-27; scores accumulated in fp32 over 36
        steps of 16 products, each off by at most 2^-23 of the magnitudes' sum; q_rope times the ratio
        of the scales in FP16 (2^-11) where that is no power of two; exponentials and sums in fp32,
        2^-20 in all; the bf16 result, 2^-8 (half a step) of itself."""
        out = np.zeros((self.num_q, self.H, 512))
        lse = np.zeros((self.num_q, self.H))
        tol, ltol = np.zeros_like(out), np.zeros_like(lse)
        f = lambda a: f32_from_bf16(a).astype(np.float64)
        exact_rope = np.log2(self.rope_scale / (self.latent_scale if self.fmt == FP8 else 1)) % 1 == 0
        for s in range(self.S):
            lat, rope, ok = self.keys(s)
            base = int(self.lens[s]) - int(self.new[s])
            for i in range(int(self.new[s])):
                t = int(self.cu[s]) + i
                if tokens is not None and t not in tokens:
                    continue
                live = np.nonzero(ok[:base + i + 1])[0]
                if live.size == 0:
                    lse[t] = -np.inf
                    continue
                k, r, ql, qr = lat[live], rope[live], f(self.ql[t]), f(self.qr[t])
                z = self.sm_scale * (ql @ k.T + qr @ r.T)
                size = abs(self.sm_scale) * (np.abs(ql) @ np.abs(k).T + np.abs(qr) @ np.abs(r).T)
                dz = size * 37 * 2.0 ** -23
                if not exact_rope:
                    dz += abs(self.sm_scale) * (np.abs(qr) @ np.abs(r).T) * 2.0 ** -11
                top = z.max(1, keepdims=True)
                e = np.exp(z - top)
                tot = e.sum(1, keepdims=True)
                w = e / tot
                out[t] = w @ k
                lse[t] = (top + np.log(tot))[:, 0]
                ltol[t] = dz.max(1) + 2.0 ** -20 * (1 + np.abs(lse[t]))
                dw = w * (2.0 ** -11 + 2 * dz + 2.0 ** -20) + 2.0 ** -27 / tot
                tol[t] = dw @ np.abs(k) + 1e-30
        return out, lse, tol, ltol

    def device(self, extra_rows=0):
        import torch
        d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")
        bf = lambda a: d(a).view(torch.bfloat16)
        return [bf(self.ql), bf(self.qr), d(self.cu), d(self.table), d(self.lens), self.page, d(self.pool).view(-1),
                self.blocks, self.stride, self.fmt, self.sm_scale, self.latent_scale, self.rope_scale]

    def check(self, out, lse, out_fp32=False, ref=None, tokens=None):
        """Results on the device against the reference; rows that are not checked are ignored."""
        ref = ref or self.reference(tokens)
        o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
        rows = np.arange(self.n) if tokens is None else np.array(sorted(tokens))
        for t in rows:
            bound = ref[2][t] + (0 if out_fp32 else 2.0 ** -8) * (np.abs(ref[0][t]) + ref[2][t])
            err = np.abs(o[t] - ref[0][t])
            assert (err <= bound).all(), (t, float((err / bound).max()), np.argwhere(~(err <= bound))[:4].tolist())
            empty = np.isneginf(ref[1][t])
            assert np.array_equal(np.isneginf(z[t]), empty), t
            lerr = np.abs(np.where(empty, 0, z[t]) - np.where(empty, 0, ref[1][t]))
            assert (lerr <= ref[3][t]).all(), (t, float(lerr.max()))
