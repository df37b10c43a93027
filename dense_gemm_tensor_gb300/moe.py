"""A mixture-of-experts block from the package's operators, and a command that
runs and times it (synthetic seeded weights and rows): a serving pass (prefill
or single tokens, 16-bit or with 8-bit rows and expert weights) or a training
step with the gradients of all weights and of the input.

    python -m dense_gemm_tensor_gb300.moe --tokens 8192
    python -m dense_gemm_tensor_gb300.moe --tokens 16 --experts 64 --dtype e4m3
    python -m dense_gemm_tensor_gb300.moe --tokens 8192 --train
"""

from __future__ import annotations

import argparse
from typing import NamedTuple

import torch

from . import build, experts, gemm
from .gemm import GEMM_B_K_MAJOR, GEMM_B_ROW_MAJOR


class Saved(NamedTuple):
    """What the backward pass needs of the forward one."""
    norm: experts.Norm
    logits: torch.Tensor
    routing: experts.Routing
    up: torch.Tensor      # slots x 2F, the gate's and the value's halves
    inner: torch.Tensor   # slots x F, silu(gate) * value
    z: torch.Tensor       # slots x H


class Grads(NamedTuple):
    x: torch.Tensor       # of the input and of the residual alike
    norm: torch.Tensor
    router: torch.Tensor
    up: torch.Tensor
    down: torch.Tensor


class MoeBlock:
    """y = h + sum over the k chosen experts of w_e * down_e(silu(gate_e(n)) * value_e(n)),
    h = x + residual, n = rms_norm(h), the weights w from the router's softmax of n . router.

    Weights: ``norm`` (H), ``router`` (H x experts), ``up`` (experts x 2F x H:
    the gate's F rows, then the value's), ``down`` (experts x H x F), float16 or
    bfloat16. ``up8``/``up8_scale`` (``quantize``): ``up`` in float8_e4m3fn with
    a scale per row, which serving then takes with 8-bit rows of n."""

    def __init__(self, norm, router, up, down, k: int, up8=None, up8_scale=None):
        self.norm, self.router, self.up, self.down, self.k = norm, router, up, down, k
        self.up8, self.up8_scale = up8, up8_scale

    @classmethod
    def random(cls, hidden: int, inner: int, n_experts: int, k: int, dtype=torch.bfloat16, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def draw(*shape, std):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

        return cls(1 + draw(hidden, std=0.1), draw(hidden, n_experts, std=hidden ** -0.5),
                   draw(n_experts, 2 * inner, hidden, std=hidden ** -0.5),
                   draw(n_experts, hidden, inner, std=inner ** -0.5), k)

    def quantize(self) -> "MoeBlock":
        """The same block with ``up`` in 8 bits as well (one scale per output column)."""
        scale = self.up.float().abs().amax(dim=2).clamp_min(1e-12) / 448.0
        up8 = (self.up.float() / scale[..., None]).to(torch.float8_e4m3fn)
        return MoeBlock(self.norm, self.router, self.up, self.down, self.k, up8, scale.contiguous())

    def serve(self, x: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        """The block's output for T x H rows; six to nine launches."""
        n = experts.rms_norm(x, self.norm, residual)
        r = experts.route(gemm.matmul(n.y, self.router), self.k)
        if self.up8 is None:
            a = experts.expert_matmul(n.y, self.up, r.offsets, r.rows, layout=GEMM_B_K_MAJOR, activation="silu_gated")
        else:
            n8 = experts.rms_norm(n.h, self.norm, out_dtype=torch.float8_e4m3fn)
            a = experts.expert_matmul(n8.y, self.up8, r.offsets, r.rows, layout=GEMM_B_K_MAJOR, a_scale=n8.scale,
                                      w_scale=self.up8_scale, activation="silu_gated")
        z = experts.expert_matmul(a, self.down, r.offsets, layout=GEMM_B_K_MAJOR)
        return experts.combine(z, r.slots, r.weights, residual=n.h)

    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        """(output, what ``backward`` needs): the 16-bit block, the gate's product kept. The activation
        and its gradient are elementary torch operations in fp32: no operator of this package has them."""
        n = experts.rms_norm(x, self.norm, residual)
        logits = gemm.matmul(n.y, self.router)
        r = experts.route(logits, self.k)
        up = experts.expert_matmul(n.y, self.up, r.offsets, r.rows, layout=GEMM_B_K_MAJOR)
        gate, value = up.chunk(2, dim=1)
        inner = (torch.nn.functional.silu(gate.float()) * value.float()).to(up.dtype)
        z = experts.expert_matmul(inner, self.down, r.offsets, layout=GEMM_B_K_MAJOR)
        return experts.combine(z, r.slots, r.weights, residual=n.h), Saved(n, logits, r, up, inner, z)

    def backward(self, dy: torch.Tensor, s: Saved) -> Grads:
        """The gradients from the output's."""
        r = s.routing
        dz, dw = experts.combine_backward(dy, s.z, r.slots, r.weights, r.offsets)
        d_down = experts.expert_weight_grad(s.inner, dz, r.offsets, layout=GEMM_B_K_MAJOR)
        d_inner = experts.expert_matmul(dz, self.down, r.offsets, layout=GEMM_B_ROW_MAJOR).float()
        gate, value = (t.float() for t in s.up.chunk(2, dim=1))
        sig = torch.sigmoid(gate)
        d_up_rows = torch.cat((d_inner * value * sig * (1 + gate * (1 - sig)), d_inner * gate * sig),
                              dim=1).to(s.up.dtype)
        d_up = experts.expert_weight_grad(s.norm.y, d_up_rows, r.offsets, r.rows, layout=GEMM_B_K_MAJOR)
        d_slots = experts.expert_matmul(d_up_rows, self.up, r.offsets, layout=GEMM_B_ROW_MAJOR)
        d_logits = experts.route_backward(dw, s.logits, r.ids)
        d_router = gemm.matmul(s.norm.y.t().contiguous(), d_logits)
        dn = experts.combine(d_slots, r.slots, residual=gemm.matmul(d_logits, self.router, layout=GEMM_B_K_MAJOR))
        dx, d_norm = experts.rms_norm_backward(dn, s.norm.h, self.norm, s.norm.rstd, dh=dy)
        return Grads(dx, d_norm, d_router, d_up, d_down)


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=" ".join(__doc__.split("\n\n")[0].split()))
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=2048, help="an expert's inner width F")
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--k", type=int, default=2, help="experts a token")
    ap.add_argument("--dtype", default="bf16", choices=("bf16", "f16", "e4m3"))
    ap.add_argument("--train", action="store_true", help="forward and backward instead of a serving pass")
    ap.add_argument("--iters", type=int, default=20)
    args = ap.parse_args(argv)
    if args.train and args.dtype == "e4m3":
        ap.error("--train takes bf16 or f16")
    build.build()
    dtype = torch.float16 if args.dtype == "f16" else torch.bfloat16
    block = MoeBlock.random(args.hidden, args.inner, args.experts, args.k, dtype)
    if args.dtype == "e4m3":
        block = block.quantize()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual, dy = (torch.randn(args.tokens, args.hidden, generator=g, device="cuda").to(dtype) for _ in range(3))

    def step():
        if args.train:
            y, saved = block.forward(x, residual)
            return block.backward(dy, saved)
        return block.serve(x, residual)

    for _ in range(3):
        step()
    before = gemm.launch_count()
    step()
    launches = gemm.launch_count() - before
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()  # single tokens: the launches' cost on the host would hide the kernels'
    with torch.cuda.graph(graph):
        step()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    torch.cuda.synchronize()
    e0.record()
    for _ in range(args.iters):
        graph.replay()
    e1.record()
    torch.cuda.synchronize()
    ms = e0.elapsed_time(e1) / max(args.iters, 1)
    flops = 2.0 * args.tokens * args.k * args.hidden * 3 * args.inner * (3 if args.train else 1)
    print(f"{args.dtype} {'training step' if args.train else 'serving pass'}, {args.tokens} tokens x {args.hidden}, "
          f"{args.k} of {args.experts} experts of inner width {args.inner}: {launches} launches of the library, {ms * 1e3:.1f} us, "
          f"{args.tokens / ms * 1e3:.0f} tokens/s, {flops / ms / 1e9:.1f} TFLOP/s in the experts")


if __name__ == "__main__":
    main()
