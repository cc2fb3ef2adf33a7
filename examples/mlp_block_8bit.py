"""A transformer MLP block trained with 8-bit activation checkpoints.

    h = x + residual;  n = LayerNorm(h);  a = GELU(n W1^T + b1);  out = a W2^T + b2 + h

Between the forward and the backward pass the block keeps, instead of the bf16
tensors n and u = n W1^T + b1, the records of the normalised rows and of u: 8.5
bits a value at block 128.  The layer norm's gradient and the first weight
gradient read the same records (scale and shift turn the normalised rows into
n), and GELU's gradient gives a again for the second weight gradient.

    python examples/mlp_block_8bit.py            # trains a small block, prints the loss and the memory kept

The linear layers are torch matrix products in bf16.  The block has first
derivatives only: its gradients come from the records, outside autograd.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_compression_tensor_gb300 as taco  # noqa: E402


class MlpBlock(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gamma, beta, w1, b1, w2, b2, block, code):
        norm = taco.layernorm(x, gamma, beta, residual=residual, checkpoint=True, block=block, code=code)
        act = taco.gelu(norm.y @ w1.t(), b1, block=block, code=code)
        ctx.save_for_backward(norm.packed, norm.rstd, act.packed, gamma, beta, w1, w2)
        ctx.options = block, code, b1.dtype, b2.dtype
        return act.y @ w2.t() + b2 + norm.summed

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        xhat, rstd, u, gamma, beta, w1, w2 = ctx.saved_tensors
        block, code, b1_dtype, b2_dtype = ctx.options
        dout = dout.contiguous()
        rows = dout.reshape(-1, dout.shape[-1])
        db2 = rows.float().sum(0).to(b2_dtype)
        act = taco.gelu_backward(dout @ w2, u, bias_dtype=torch.float32, recompute=True, block=block, code=code)
        dw2 = rows.t() @ act.y.reshape(-1, act.y.shape[-1])
        dw1 = taco.weight_grad(act.dx, xhat, w1.shape[1], scale=gamma, shift=beta, dy_sum=act.dbias, dtype=w1.dtype,
                               block=block, code=code)
        norm = taco.layernorm_backward(act.dx @ w1, rstd, gamma, packed=xhat, dsummed=dout, block=block, code=code)
        return (norm.dx, norm.dx, norm.dweight, norm.dbias, dw1, act.dbias.to(b1_dtype), dw2.to(w2.dtype), db2, None, None)


def mlp_block(x, residual, gamma, beta, w1, b1, w2, b2, block=128, code="e4m3"):
    """The block's output; differentiable in the first eight arguments."""
    return MlpBlock.apply(x, residual, gamma, beta, w1, b1, w2, b2, block, code)


def parameters(hidden, inner, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device=device)
    f32, bf16 = torch.float32, torch.bfloat16
    made = [1 + 0.1 * normal(hidden), 0.1 * normal(hidden), normal(inner, hidden) * hidden ** -0.5, 0.1 * normal(inner),
            normal(hidden, inner) * inner ** -0.5, 0.1 * normal(hidden)]
    return [p.to(t).requires_grad_() for p, t in zip(made, (f32, f32, bf16, f32, bf16, bf16))]


def main(tokens=2048, hidden=1024, steps=20):
    params = parameters(hidden, 4 * hidden)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    residual = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    for step in range(steps):
        out = mlp_block(x, residual, *params)
        loss = (out.float() - target.float()).square().mean()
        grads = torch.autograd.grad(loss, params)
        with torch.no_grad():
            for p, d in zip(params, grads):
                p -= 2.0 * d
        if step % 5 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {loss.item():.5f}")
    kept = taco.compressed_bytes(tokens, hidden) + taco.compressed_bytes(tokens, 4 * hidden) + 4 * tokens
    print(f"kept for the backward pass: {kept / 1e6:.2f} MB, in bf16 {2 * tokens * 5 * hidden / 1e6:.2f} MB")
    assert taco.device_status() == 0


if __name__ == "__main__":
    main()
