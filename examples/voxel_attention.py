"""A voxel block that mixes convolution and attention, trained for a few steps on synthetic shells.

One step: 3x3x3 submanifold convolution -> queries, keys and values of the voxels -> norm of queries and keys with the
voxel coordinates' rotation (three axes) -> self attention inside each sample -> cross attention to an encoder's states
(padded, with a mask) -> one pooled token per sample reading its voxels -> squared error, backward, gradient step.

    python examples/voxel_attention.py [--config 2] [--steps 5] [--dtype bf16]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import sparse_submanifold_convolution_amd as ssc  # noqa: E402
from sparse_submanifold_convolution_amd import workloads as WL  # noqa: E402

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class VoxelBlock(torch.nn.Module):
    """Parameters of the block; `width` channels in `heads` heads, encoder states of `states` channels."""

    def __init__(self, width: int, heads: int, states: int, dtype: torch.dtype, device):
        super().__init__()
        self.heads, self.dim = heads, width // heads
        g = torch.Generator(device=device).manual_seed(0)

        def weight(*shape, fan):
            w = torch.randn(*shape, generator=g, device=device) * fan ** -0.5
            return torch.nn.Parameter(w.to(dtype))

        def ones():
            return torch.nn.Parameter(torch.ones(heads, self.dim, dtype=dtype, device=device))

        self.conv = weight(27, width, width, fan=9 * width)
        self.qkv = weight(width, 3 * width, fan=width)
        self.q_cross = weight(width, width, fan=width)
        self.kv_cross = weight(states, 2 * width, fan=states)
        self.pool = weight(1, heads, self.dim, fan=1)
        self.norms = torch.nn.ParameterList([ones() for _ in range(4)])
        pairs = self.dim // 2
        self.table = ssc.rope_table((pairs - 2 * (pairs // 3), pairs // 3, pairs // 3), device=device)

    def forward(self, feats, plan, coords, offsets, states, state_offsets, state_mask, pool_offsets):
        n, h, d = feats.shape[0], self.heads, self.dim
        x = feats + ssc.subm_conv3d(feats, plan, self.conv)
        # self attention: the packed projection's heads are read where they lie
        qkv = (x @ self.qkv).view(n, 3 * h, d)
        q, k = ssc.qk_norm_rope(qkv[:, :h], qkv[:, h:2 * h], coords[:, 1:], self.table, self.norms[0], self.norms[1])
        x = x + ssc.cross_attention(q, k, qkv[:, 2 * h:], offsets, offsets).reshape(n, h * d)
        # cross attention to the encoder's states, which have no voxel positions: norm only
        kv = (states @ self.kv_cross).view(-1, 2 * h, d)
        q, _ = ssc.qk_norm_rope((x @ self.q_cross).view(n, h, d), None, q_weight=self.norms[2])
        _, k = ssc.qk_norm_rope(None, kv[:, :h], k_weight=self.norms[3])
        x = x + ssc.cross_attention(q, k, kv[:, h:], offsets, state_offsets, state_mask).reshape(n, h * d)
        # one learned query per sample reads all of its voxels
        batch = pool_offsets.numel() - 1
        rows = x.view(n, h, d)
        token = ssc.cross_attention(self.pool.expand(batch, h, d), rows, rows, pool_offsets, offsets)
        return x, token.reshape(batch, h * d)


def inputs(config: int, states_len: int, states_width: int, dtype: torch.dtype, device):
    """Voxels of one of the benchmark's workloads, rows in z-order (so grouped by sample), and padded encoder states."""
    w = WL.make_workload(config)
    coords = torch.from_numpy(w.coords).to(device)
    order = torch.argsort(ssc.encode_seq(coords, w.shape))
    coords = coords[order].contiguous()
    feats = w.feats.to(device)[order].to(dtype).contiguous()
    batch = w.shape[0]
    g = torch.Generator(device=device).manual_seed(1)
    states = torch.randn(batch * states_len, states_width, generator=g, device=device).to(dtype)
    used = torch.randint(states_len // 2, states_len + 1, (batch, 1), generator=g, device=device)
    mask = (torch.arange(states_len, device=device) < used).reshape(-1)
    state_offsets = torch.arange(batch + 1, dtype=torch.int32, device=device) * states_len
    return {"plan": ssc.build_neighbor_map(coords, w.shape), "coords": coords, "feats": feats,
            "offsets": ssc.row_offsets(coords, batch), "states": states, "state_offsets": state_offsets,
            "state_mask": mask, "pool_offsets": torch.arange(batch + 1, dtype=torch.int32, device=device)}


def train(config: int = 2, steps: int = 5, dtype: str = "bf16", lr: float = 0.2, report=print):
    """Runs the steps and returns their losses."""
    device = torch.device("cuda:0")
    data = inputs(config, 77, 48, DTYPES[dtype], device)
    width = data["feats"].shape[1]
    block = VoxelBlock(width, max(1, width // 32), 48, DTYPES[dtype], device)
    g = torch.Generator(device=device).manual_seed(2)
    target = torch.randn(data["pool_offsets"].numel() - 1, width, generator=g, device=device)
    losses = []
    for step in range(steps):
        x, token = block(**data)
        loss = ((token.float() - target) ** 2).mean() + 0.01 * (x.float() ** 2).mean()
        loss.backward()
        with torch.no_grad():
            for p in block.parameters():
                p.sub_((lr * p.grad.float()).to(p.dtype))
                p.grad = None
        losses.append(loss.item())
        report(f"step {step}: {data['feats'].shape[0]} voxels, loss {losses[-1]:.4f}", flush=True)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--config", type=int, default=2)
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--dtype", choices=sorted(DTYPES), default="bf16")
    a = ap.parse_args()
    train(a.config, a.steps, a.dtype)
