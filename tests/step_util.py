"""Builds a serving step on the GPU and its 64-bit expectation (used by test_gpu_step.py)."""
from __future__ import annotations

import numpy as np
import torch

from oracle import step_oracle as so
from position_free_kv_amd import abi, step

TYPES = {abi.BF16: torch.bfloat16, abi.F32: torch.float32}
HALF = {abi.BF16: torch.finfo(torch.bfloat16).eps / 2, abi.F32: torch.finfo(torch.float32).eps / 2}
E32 = 2.0 ** -24


class Case:
    """requests: (prefix or -1, own tokens, queries[, flags]); prefixes: token counts."""

    def __init__(self, *, family=abi.GQA, dtype=abi.BF16, heads=4, kv_heads=2, head_dim=64, latent=0, rope=0, layers=2,
                 page=16, prefixes=(), requests=(), seed=0, spare=3, pad_layer=0, offset=0, base=1e4, pairing=abi.NEOX,
                 sections=(0, 0, 0), garbage=float("nan"), device="cuda"):
        rng = np.random.default_rng([seed, 5])
        self.rng, self.dtype, self.page, self.layers, self.heads, self.family = rng, dtype, page, layers, heads, family
        self.hkv, self.dk = (kv_heads, head_dim) if family == abi.GQA else (1, latent + rope)
        self.dv = head_dim if family == abi.GQA else latent
        self.F = self.hkv * self.dk
        self.g = heads // self.hkv if heads else 0
        self.latent, self.d_rot, self.base, self.pairing, self.sections = latent, head_dim if family == abi.GQA else rope, base, pairing, sections
        self.requests, self.prefix_tokens = [tuple(r) + (0,) * (4 - len(r)) for r in requests], list(prefixes)
        self.lay = abi.make_layout(family, dtype, layers, num_kv_heads=kv_heads if family == abi.GQA else 0,
                                   head_dim=head_dim if family == abi.GQA else 0, latent_dim=latent, rope_dim=rope,
                                   pairing=pairing, rope_base=base, page_size=page, mrope_section=sections)
        # tables: every prefix and request on pages of its own, in random order, starting inside a page
        self.slot0 = [int(rng.integers(0, page)) for _ in range(len(prefixes) + len(requests))]
        lens = list(prefixes) + [r[1] for r in self.requests]
        need = [-(-(s + n) // page) if n else 0 for s, n in zip(self.slot0, lens)]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        cut = np.cumsum([0] + need)
        self.tables = [order[a:b].copy() for a, b in zip(cut[:-1], cut[1:])]
        self.rows = [so.slots(t, s, n, page) if n else np.zeros(0, np.int64) for t, s, n in zip(self.tables, self.slot0, lens)]
        # pools: garbage everywhere, then the rows in use
        t = TYPES[dtype]
        tensors = 2 if family == abi.GQA else 1
        per_layer = self.pages * page * self.F + pad_layer
        self.flat = [torch.full((layers * per_layer + offset,), garbage, dtype=t, device=device) for _ in range(tensors)]
        self.pools = [f[offset:].as_strided((layers, self.pages * page, self.F), (per_layer, self.F, 1)) for f in self.flat]
        used = np.concatenate(self.rows) if self.rows else np.zeros(0, np.int64)
        for p in self.pools:
            p[:, torch.from_numpy(used).to(device)] = self.draw(layers, used.size, self.F).to(device)
        self.pool = abi.make_pool(self.pools[0], self.pools[-1] if tensors == 2 else None, self.pages, per_layer)
        self.n = sum(r[2] for r in self.requests)
        self.q = self.draw(layers, self.n, heads * self.dk).to(device) if heads else None
        self.device = device

    def draw(self, *shape):
        x = torch.from_numpy(self.rng.standard_normal(shape).astype(np.float32))
        return x.to(TYPES[self.dtype])

    def step(self, flags, **more):
        np_ = len(self.prefix_tokens)
        return step.Step(num_q_heads=self.heads, block_tables=[t if t.size else None for t in self.tables[np_:]],
                         slot0=self.slot0[np_:], num_tokens=[r[1] for r in self.requests],
                         num_queries=[r[2] for r in self.requests], prefix=[r[0] for r in self.requests],
                         request_flags=[r[3] for r in self.requests],
                         prefixes=[dict(block_table=t, slot0=s, num_tokens=n) for t, s, n in
                                   zip(self.tables[:np_], self.slot0[:np_], self.prefix_tokens)], flags=flags, **more)

    def workspace(self, s):
        size = step.workspace_bytes(self.lay, s)
        assert size > 0
        return torch.empty(size, dtype=torch.uint8, device=self.device)

    # ---------------------------------------------------------------- attention
    def attend(self, scale, stream=None):
        s = self.step(step.ATTEND)
        ws = self.workspace(s)
        plan = step.upload(self.lay, s, self.pool, ws, stream=stream)
        out = torch.full((self.layers, self.n, self.heads * self.dv), 7.0, dtype=TYPES[self.dtype], device=self.device)
        lse = torch.full((self.layers, self.n, self.heads), 7.0, device=self.device)
        for layer in range(self.layers):
            step.attend(plan, layer, self.q[layer], out[layer], scale, lse=lse[layer], stream=stream)
        return out, lse

    def expect_attend(self, layer, scale):
        """(out, tolerance, lse, tolerance) in 64 bits."""
        f64 = [p[layer].double().cpu().numpy() for p in self.pools]
        q = self.q[layer].double().cpu().numpy().reshape(self.n, self.heads, self.dk)
        out, tol = np.zeros((self.n, self.heads, self.dv)), np.zeros((self.n, self.heads, self.dv))
        lse, ltol = np.zeros((self.n, self.heads)), np.zeros((self.n, self.heads))
        n0 = 0
        np_ = len(self.prefix_tokens)
        for r, (pre, own, nq, flags) in enumerate(self.requests):
            head = self.rows[pre] if pre >= 0 else np.zeros(0, np.int64)
            at = np.concatenate([head, self.rows[np_ + r]])
            last = np.full(nq, at.size - 1) if flags else np.maximum(head.size + own - nq + np.arange(nq), head.size - 1)
            for h in range(self.hkv):
                k = f64[0][at, h * self.dk:(h + 1) * self.dk]
                v = f64[-1][at, h * self.dk:h * self.dk + self.dv]
                sl = slice(h * self.g, (h + 1) * self.g)
                o, z, a, terms = so.attend(q[n0:n0 + nq, sl], k, v, scale, last)
                out[n0:n0 + nq, sl], lse[n0:n0 + nq, sl] = o, z
                # Scores: dk products accumulated in fp32, the scale, its product with log2(e):
                # off by ds. A probability exp(s - m) is then off by 2 ds relative (s and the
                # maximum), and by the exponential's and the joins' own few fp32 roundings; sums
                # over at.size of them add at.size roundings at most. On the matrix cores each
                # probability is rounded to bf16 once more. The output is rounded once.
                ds = (self.dk + 8) * E32 * terms[..., None]
                rel = 2 * ds + (2 * at.size + 128) * E32 + (HALF[abi.BF16] if self.dtype == abi.BF16 else 0.0)
                # 1e-38: products of fp32 numbers below the smallest normal one may vanish
                tol[n0:n0 + nq, sl] = rel * (a + np.abs(o)) + HALF[self.dtype] * np.abs(o) + 1e-38
                seen = np.isfinite(z)
                ltol[n0:n0 + nq, sl] = ds[..., 0] + (at.size + 128) * E32 + 8 * E32 * np.where(seen, np.abs(np.where(seen, z, 0)), 0)
            n0 += nq
        return out.reshape(self.n, -1), tol.reshape(self.n, -1), lse, ltol

    def check_attend(self, scale, stream=None):
        out, lse = self.attend(scale, stream)
        torch.cuda.synchronize()
        for layer in range(self.layers):
            o, tol, z, ltol = self.expect_attend(layer, scale)
            got, gz = out[layer].double().cpu().numpy(), lse[layer].double().cpu().numpy()
            assert np.isfinite(got).all(), f"layer {layer}: {np.argwhere(~np.isfinite(got))[:4]}"
            bad = np.abs(got - o) > tol
            assert not bad.any(), (layer, np.argwhere(bad)[:4].tolist(), got[bad][:4], o[bad][:4], tol[bad][:4], int(bad.sum()))
            empty = np.isneginf(z)
            assert (np.isneginf(gz) == empty).all()
            off = np.abs(np.where(empty, 0, gz) - np.where(empty, 0, z))
            assert (off <= ltol).all(), (layer, float((off - ltol).max()))
        return out, lse
