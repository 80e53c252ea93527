"""A mixture-of-experts block as a transformer layer has it, on the library's entry points:

    s = x + residual;  n = RMSNorm(s);  logits = n Wr^T;  top experts and weights of each token
    y = s + sum_j w_j Expert_{e_j}(n),  Expert(n) = W2 SwiGLU(W1 n)

``ExpertBlock.decode`` takes up to 64 tokens: norm, router product, routing, and the whole
expert layer straight from the ids.  ``forward`` / ``backward`` take any number: the routing's
plan orders the tokens by expert for the grouped MLP, and every gradient comes from the
library; only rows are moved (gathered, scattered, weighted) by torch indexing.  Features,
ffn and experts are multiples of 8.

    python examples/expert_block.py        # on an MI355X: both paths agree, time of each
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import grouped_gemm_gl_amd as gl  # noqa: E402


class ExpertBlock:
    def __init__(self, features: int, ffn: int, experts: int, top_k: int, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.E, self.k, self.F, self.eps, self.dtype = experts, top_k, ffn, 1e-6, dtype
        self.gamma = 1 + 0.1 * r(features)
        self.wr = (r(1, experts, features) * features ** -0.5).to(dtype)
        self.w1 = (r(experts, 2 * ffn, features) * features ** -0.5).to(dtype)
        self.w2 = (r(experts, features, ffn) * ffn ** -0.5).to(dtype)
        self.one, self.plan = gl.new_workspace(1, device), gl.new_workspace(experts, device)

    def _new(self, *shape, dtype=None):
        return torch.empty(*shape, dtype=dtype or self.dtype, device=self.gamma.device)

    def _norm_and_route(self, x, residual, with_plan):
        T, C = x.shape
        c = {"s": self._new(T, C), "n": self._new(T, C), "logits": self._new(T, self.E),
             "ids": self._new(T, self.k, dtype=torch.int32), "weights": self._new(T, self.k, dtype=torch.float32)}
        gl.gl_rmsnorm_forward(x, self.gamma, self.eps, residual=residual, h=c["s"], y=c["n"])
        gl.gl_offsets(torch.full((1,), T, dtype=torch.int64, device=x.device), T, self.one)
        gl.gl_forward(c["n"], self.wr, c["logits"], self.one)
        kw = {}
        if with_plan:
            c["m_splits"] = self._new(self.E, dtype=torch.int64)
            c["row_index"], c["slot_index"] = self._new(T, self.k, dtype=torch.int32), self._new(T * self.k, dtype=torch.int32)
            kw = {n: c[n] for n in ("m_splits", "row_index", "slot_index")}
            kw["workspace"] = self._new(gl.gl_route_workspace_size(T, self.E), dtype=torch.uint8)
        gl.gl_route_forward(c["logits"], c["ids"], c["weights"], **kw)
        return c

    def decode(self, x, residual):
        """y [T, features] of up to gl.MOE_MAX_TOKENS tokens."""
        c = self._norm_and_route(x, residual, with_plan=False)
        ws = self._new(gl.gl_moe_few_tokens_workspace_size(x.shape[0], self.k, self.E, self.F), dtype=torch.uint8)
        return gl.gl_moe_few_tokens(c["n"], c["ids"], c["weights"], self.w1, self.w2, c["s"], ws, residual=c["s"])

    def forward(self, x, residual):
        """y and what the backward needs."""
        T, C = x.shape
        c = self._norm_and_route(x, residual, with_plan=True)
        rows = T * self.k
        gl.gl_offsets(c["m_splits"], rows, self.plan)
        c["token"] = torch.div(c["slot_index"], self.k, rounding_mode="floor").long()
        c["rows"] = c["n"][c["token"]]
        c["h"], c["a"], c["z"] = self._new(rows, 2 * self.F), self._new(rows, self.F), self._new(rows, C)
        gl.gl_grouped_mlp_forward(c["rows"], self.w1, self.w2, c["h"], c["a"], c["z"], self.plan)
        z = c["z"][c["row_index"].long()]  # [T, top_k, C]
        y = c["s"].float() + (z.float() * c["weights"][..., None]).sum(1)
        return y.to(self.dtype), c

    def backward(self, dy, c):
        """Gradients of x (and the residual alike), gamma and the weights."""
        T, C = dy.shape
        z = c["z"][c["row_index"].long()].float()
        dweights = (z * dy.float()[:, None]).sum(-1)
        w_row = c["weights"].reshape(-1)[c["slot_index"].long()]
        dz = (dy.float()[c["token"]] * w_row[:, None]).to(self.dtype)
        drows, da, dh = torch.empty_like(c["rows"]), torch.empty_like(c["a"]), torch.empty_like(c["h"])
        dw1, dw2 = self._new(*self.w1.shape, dtype=torch.float32), self._new(*self.w2.shape, dtype=torch.float32)
        gl.gl_grouped_mlp_backward(c["rows"], self.w1, self.w2, c["h"], c["a"], dz, da, dh, drows, dw1, dw2, self.plan)
        dlogits = torch.empty_like(c["logits"])
        gl.gl_route_backward(c["logits"], c["ids"], dweights, dlogits)
        dn_router, dwr = self._new(T, C), self._new(*self.wr.shape, dtype=torch.float32)
        gl.gl_offsets(torch.full((1,), T, dtype=torch.int64, device=dy.device), T, self.one)
        gl.gl_dgrad(dlogits, self.wr, dn_router, self.one)
        gl.gl_wgrad(c["n"], dlogits, dwr, self.one)
        dn = (drows[c["row_index"].long()].float().sum(1) + dn_router.float()).to(self.dtype)
        dx, dgamma = self._new(T, C), self._new(C, dtype=torch.float32)
        ws = self._new(gl.gl_rmsnorm_workspace_size(T, C), dtype=torch.uint8)
        gl.gl_rmsnorm_backward(dn, c["s"], self.gamma, self.eps, dx, dh=dy, dgamma=dgamma, workspace=ws)
        return {"x": dx, "gamma": dgamma, "wr": dwr, "w1": dw1, "w2": dw2}


def main():
    block = ExpertBlock(features=2048, ffn=768, experts=64, top_k=8)
    g = torch.Generator(device="cuda").manual_seed(1)
    for T in (1, 16, 64, 4096):
        x, residual = (torch.randn(T, 2048, generator=g, device="cuda").bfloat16() for _ in range(2))
        calls = {"forward": lambda: block.forward(x, residual)[0]}
        if T <= gl.MOE_MAX_TOKENS:
            calls["decode"] = lambda: block.decode(x, residual)
        else:
            dy = torch.randn(T, 2048, generator=g, device="cuda").bfloat16()
            calls["forward and backward"] = lambda: block.backward(dy, block.forward(x, residual)[1])
        out = {}
        for name, call in calls.items():
            for _ in range(3):
                out[name] = call()
            torch.cuda.synchronize()
            t = time.perf_counter()
            for _ in range(20):
                call()
            torch.cuda.synchronize()
            print(f"{T:5d} tokens, {name}: {(time.perf_counter() - t) / 20 * 1e6:.0f} us", flush=True)
        if "decode" in out:
            off = (out["decode"].float() - out["forward"].float()).norm() / out["forward"].float().norm()
            print(f"{T:5d} tokens: decode and forward differ by {off:.1e} of their norm", flush=True)


if __name__ == "__main__":
    main()
