"""A gated feed-forward block trained with 8-bit activation checkpoints.

    h = x + residual;  n = RMSNorm(h);  a = silu(n Wg^T) * (n Wu^T);  out = a Wd^T + h

Both projections, the activation and the product are one kernel, W = [Wg; Wu].
Between the forward and the backward pass the block keeps, instead of the bf16
tensors n and n W^T, the records of the normalised rows and of both
projections: 8.5 bits a value at block 128.  The backward pass makes the
projections' gradient dz and a again from the records, the input's gradient dz W,
and the weight gradient dz^T n from the normalised rows (scale turns them
into n); the down projection is a torch matrix product in bf16.

    python examples/gated_block_8bit.py            # trains a small block, prints the loss and the memory kept

The block has first derivatives only: its gradients come from the records,
outside autograd.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_compression_tensor_gb300 as taco  # noqa: E402


class GatedBlock(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gamma, w, wd, activation, block, code):
        norm = taco.rmsnorm(x, gamma, residual=residual, checkpoint=True, block=block, code=code)
        gated = taco.gated_linear(norm.y, w, activation=activation, checkpoint=True, block=block, code=code)
        ctx.save_for_backward(norm.packed, norm.rstd, gated.packed, gamma, w, wd)
        ctx.options = activation, block, code
        return gated.y @ wd.t() + norm.summed

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        xhat, rstd, z, gamma, w, wd = ctx.saved_tensors
        activation, block, code = ctx.options
        dout = dout.contiguous()
        rows = dout.reshape(-1, dout.shape[-1])
        gated = taco.gated_linear_backward(dout @ wd, z, w, activation=activation, recompute=True, block=block, code=code)
        dwd = rows.t() @ gated.y.reshape(-1, gated.y.shape[-1])
        dw = taco.weight_grad(gated.dz, xhat, w.shape[1], scale=gamma, dtype=w.dtype, block=block, code=code)
        norm = taco.rmsnorm_backward(gated.dx, rstd, gamma, packed=xhat, dsummed=dout, block=block, code=code)
        return norm.dx, norm.dx, norm.dweight, dw, dwd.to(wd.dtype), None, None, None


def gated_block(x, residual, gamma, w, wd, activation="silu", block=128, code="e4m3"):
    """The block's output; differentiable in the first five arguments."""
    return GatedBlock.apply(x, residual, gamma, w, wd, activation, block, code)


def parameters(hidden, inner, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device=device)
    made = [1 + 0.1 * normal(hidden), normal(2 * inner, hidden) * hidden ** -0.5, normal(hidden, inner) * inner ** -0.5]
    return [p.to(t).requires_grad_() for p, t in zip(made, (torch.float32, torch.bfloat16, torch.bfloat16))]


def main(tokens=2048, hidden=1024, inner=2688, steps=20):
    params = parameters(hidden, inner)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual, target = (torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    for step in range(steps):
        out = gated_block(x, residual, *params)
        loss = (out.float() - target.float()).square().mean()
        grads = torch.autograd.grad(loss, params)
        with torch.no_grad():
            for p, d in zip(params, grads):
                p -= 2.0 * d
        if step % 5 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {loss.item():.5f}")
    kept = taco.compressed_bytes(tokens, hidden) + taco.compressed_bytes(tokens, 2 * inner) + 4 * tokens
    print(f"kept for the backward pass: {kept / 1e6:.2f} MB, in bf16 {2 * tokens * (hidden + 2 * inner) / 1e6:.2f} MB")
    assert taco.device_status() == 0


if __name__ == "__main__":
    main()
