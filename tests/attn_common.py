"""Paged-cache problems for the GPU tests: seeded inputs on the CPU, the library's calls, and error bounds."""

import numpy as np
import torch

from hybrid_linear_attention_gated_gb300 import hla, inputs

BF16, F32, I32, FP8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def bits(t):
    """The tensor's bytes (equality of bits, NaN included)."""
    return t.contiguous().view(torch.uint8)


class Problem:
    """A cache whose pages hold N(0, 1) keys and values up to each sequence's past + T tokens and, everywhere else,
    NaN (so that a read of a place that holds no key shows)."""

    def __init__(self, dev, past, T=1, H=8, Hkv=2, d=128, page=64, dtype=hla.HLA_BF16, seed=0, spare=2, max_blocks=None,
                 poison=True, k_std=1.0):
        self.dev, self.past, self.B, self.T, self.H, self.Hkv, self.d, self.page = dev, list(past), len(past), T, H, Hkv, d, page
        g = inputs.generator(seed)
        need = [-(-(p + T) // page) if p >= 0 else 0 for p in self.past]
        self.n_pages = sum(need) + spare
        self.max_blocks = max_blocks or max(need + [1])
        order = torch.randperm(self.n_pages, generator=g).to(I32)
        self.table = torch.full((self.B, self.max_blocks), -1, dtype=I32)
        at = 0
        for b, n in enumerate(need):
            m = min(n, self.max_blocks)
            self.table[b, :m] = order[at:at + m]
            at += n
        store = FP8 if dtype == hla.HLA_E4M3 else BF16
        unit = 24.0 if dtype == hla.HLA_E4M3 else k_std
        shape = (self.n_pages, Hkv, page, d)
        self.k = (torch.randn(shape, generator=g) * unit).to(store)
        self.v = (torch.randn(shape, generator=g) * unit).to(store)
        if poison:
            valid = torch.zeros(self.n_pages, page, dtype=torch.bool)
            for b, p in enumerate(self.past):
                for c in range(p + T if p >= 0 else 0):
                    if c // page < self.max_blocks:
                        valid[self.table[b, c // page], c % page] = True
            for x in (self.k, self.v):
                x.copy_(torch.where(valid[:, None, :, None], x.float(), float("nan")).to(store))
        self.q = torch.randn((self.B, T, H, d), generator=g).to(BF16)
        self.k_scale = self.v_scale = None
        if dtype == hla.HLA_E4M3:
            self.k_scale, self.v_scale = ((torch.rand(Hkv, generator=g) + 0.5) / 24 for _ in range(2))
        self.k_min = self.k_max = None
        self.dtype, self.scale = dtype, 1 / d ** 0.5

    # -- device side
    def upload(self):
        up = lambda t: None if t is None else t.to(self.dev)  # noqa: E731
        self.D = dict(k=up(self.k), v=up(self.v), ks=up(self.k_scale), vs=up(self.v_scale), q=up(self.q), table=up(self.table),
                      past=torch.tensor(self.past, dtype=I32, device=self.dev), lo=up(self.k_min), hi=up(self.k_max))
        D = self.D
        self.C = hla.make_kv_cache(self.dtype, self.n_pages, self.page, self.Hkv, self.d, D["k"], D["v"], D["ks"], D["vs"],
                                   D["lo"], D["hi"])
        return self

    def decode(self, o_dtype=hla.HLA_BF16, sel=None, stream=None, ws=None, o=None):
        D = self.D
        if o is None:
            o = torch.full((self.B, self.T, self.H, self.d), 7.0, dtype=BF16 if o_dtype == hla.HLA_BF16 else F32, device=self.dev)
        if sel is None:
            n = hla.attn_paged_decode_workspace_size(self.C, self.B, self.T, self.H)
            ws = torch.empty(n, dtype=torch.uint8, device=self.dev) if ws is None else ws
            hla.attn_paged_decode(self.C, self.B, self.T, self.H, self.max_blocks, D["table"], D["past"], self.scale, D["q"], o,
                                  o_dtype, ws, ws.numel(), stream)
        else:
            n = hla.attn_paged_sparse_workspace_size(self.C, self.B, self.T, self.H)
            ws = torch.empty(n, dtype=torch.uint8, device=self.dev) if ws is None else ws
            hla.attn_paged_sparse(self.C, self.B, self.T, self.H, self.max_blocks, D["table"], D["past"], sel.shape[-1], sel,
                                  self.scale, D["q"], o, o_dtype, ws, ws.numel(), stream)
        return o

    def select(self, n_select, n_first=0, n_last=0, stream=None, ws=None, sel=None):
        D = self.D
        if sel is None:
            sel = torch.full((self.B, self.T, self.Hkv, n_select), -7, dtype=I32, device=self.dev)
        n = hla.attn_select_blocks_workspace_size(self.C, self.B, self.T, self.H, self.max_blocks)
        ws = torch.empty(n, dtype=torch.uint8, device=self.dev) if ws is None else ws
        hla.attn_select_blocks(self.C, self.B, self.T, self.H, self.max_blocks, D["table"], D["past"], n_select, n_first, n_last,
                               D["q"], sel, ws, ws.numel(), stream)
        return sel

    # -- oracle side: the values that the cache stands for
    def values(self):
        k, v = self.k.double().numpy(), self.v.double().numpy()
        if self.k_scale is not None:
            k = k * self.k_scale.double().numpy()[None, :, None, None]
            v = v * self.v_scale.double().numpy()[None, :, None, None]
        return k, v


def attention_tolerance(ref, mag, n_keys, d, score_size, o_dtype, cache_dtype):
    """Elementwise bound on |o - ref|, ref exact and mag = sum of weight x |value|.

    A score is a chain of d fp32 additions whose terms' magnitudes add up to score_size: off by d 2^-23 of it, and so is, to
    first order, the weight relative to itself, twice (numerator and sum); exp2 adds 2^-21.  A weight meets V rounded by half a
    step: bf16 2^-8, fp16 (8-bit cache) 2^-11 and for weights below 2^-28 nothing; an fp32 output keeps the rounded-off part to
    the same relative precision again, twice with bf16.  The sums over keys are chains of n_keys additions: n_keys 2^-23 of mag.  The output
    rounds by 2^-8 (bf16) or 2^-24."""
    score = 2 * (d * 2.0 ** -23 * score_size + 2.0 ** -21)
    half = 2.0 ** -11 if cache_dtype == hla.HLA_E4M3 else 2.0 ** -8
    out_f32 = o_dtype == hla.HLA_F32
    weight = half ** (2 if cache_dtype == hla.HLA_E4M3 else 3) if out_f32 else half
    return (2.0 ** -24 if out_f32 else 2.0 ** -8) * np.abs(ref) + (score + weight + 2 * n_keys * 2.0 ** -23 + n_keys * 2.0 ** -28) * mag
