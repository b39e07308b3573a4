"""Pillars as tokens: a small model that is trained on frames and then asked.

Each frame's points are voxelized; a pillar's token is the mean of its points,
projected, plus the learned row of its cell (``embed``). One layer lets the
tokens of a frame attend to each other, nearer ones more (``attend``), another
mixes them along their order (``gated_scan``). Training regresses how full each
pillar is; afterwards one new token per frame attends to the frame's kept keys
and continues the recurrence from its last state, as a decoding step does.

With ``next`` it learns what comes next instead: queries and keys are turned by their
places (``rotate``), tokens mix along their order at a cost that grows with their
number alone (``decay_attend``), and each token's output is compared with the learned
rows of all cells (``row_loss``); afterwards one new token per frame continues from the
kept states and says how likely a cell is.

    python examples/pillar_tokens.py [steps] [next]
"""
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import sparse_spatial_hashing_amd as ssh  # noqa: E402
from workloads import generate, get_config  # noqa: E402


class PillarTokens(torch.nn.Module):
    def __init__(self, cells, width=64, heads=4, kv_heads=2):
        super().__init__()
        self.width, self.heads, self.kv_heads = width, heads, kv_heads
        self.head_width = width // heads
        self.cells = torch.nn.Parameter(torch.randn(cells, width) / width)
        self.features = torch.nn.Linear(4, width)
        self.qkv = torch.nn.Linear(width, (heads + 2 * kv_heads) * self.head_width, bias=False)
        self.mix = torch.nn.Linear(width, 2 * width)
        self.full = torch.nn.Linear(width, 1)
        self.register_buffer("slopes", 2.0 ** -torch.arange(1, heads + 1).float())

    def heads_of(self, x):
        """q, k and v of tokens, strided views of one product."""
        x = self.qkv(x).to(torch.bfloat16).unflatten(1, (-1, self.head_width))
        return x.split([self.heads, self.kv_heads, self.kv_heads], 1)

    def forward(self, means, ids, places, offsets):
        x = self.features(means) + ssh.embed(self.cells, ids, scale=math.sqrt(self.width))
        q, k, v = self.heads_of(x)
        seen = ssh.attend(q, k, v, q_offsets=offsets, k_offsets=offsets, cap=20.0,
                          slopes=self.slopes, q_pos=places, k_pos=places)
        x = x + seen.flatten(1).float()
        gate, value = self.mix(x).chunk(2, 1)
        mixed, state = ssh.gated_scan(gate, value, offsets)
        return self.full(x + mixed).squeeze(1), (k, v, state)

    @torch.no_grad()
    def ask(self, x, places, kept, offsets, key_places):
        """One new token per frame, x [frames, width], over what forward kept."""
        k, v, state = kept
        frames = offsets.shape[0] - 1
        one = torch.arange(frames + 1, dtype=torch.int32, device=x.device)
        q = self.heads_of(x)[0]
        seen = ssh.attend(q, k, v, q_offsets=one, k_offsets=offsets, cap=20.0, slopes=self.slopes,
                          q_pos=places, k_pos=key_places)
        x = x + seen.flatten(1).float()
        gate, value = self.mix(x).chunk(2, 1)
        mixed, state = ssh.gated_scan(gate, value, one, state=state)
        return self.full(x + mixed).squeeze(1), state


class NextPillar(torch.nn.Module):
    """Which cell the next pillar of a frame is in, from the pillars before it."""

    def __init__(self, cells, width=64, heads=4):
        super().__init__()
        self.width, self.heads = width, heads
        self.cells = torch.nn.Parameter(torch.randn(cells, width) * width ** -0.5)
        self.features = torch.nn.Linear(4, width)
        self.qkv = torch.nn.Linear(width, 3 * width, bias=False)
        self.register_buffer("decay", 2.0 ** -(1.0 + 2.0 * torch.arange(heads)))
        self.register_buffer("freqs", ssh.rotary_frequencies(width // heads, axes=2, device="cpu"))

    def forward(self, means, ids, places, offsets, state=None):
        x = self.features(means) + ssh.embed(self.cells, ids, scale=math.sqrt(self.width))
        qkv = self.qkv(x).to(torch.bfloat16).unflatten(1, (3 * self.heads, -1))
        turned = ssh.rotate(qkv[:, :2 * self.heads], places, self.freqs)
        mixed, state = ssh.decay_attend(*turned.split(self.heads, 1), qkv[:, 2 * self.heads:], self.decay, offsets,
                                        state=state)
        return (x + mixed.flatten(1).float()).to(torch.bfloat16), state

    def loss(self, x, ids):
        return ssh.row_loss(x, self.cells.to(torch.bfloat16), ids)


def frames_of(device, counts=(4168, 3000, 1200)):
    """Frames of the tiny configuration, voxelized and packed."""
    p = get_config("tiny").params
    cloud = torch.from_numpy(generate("tiny")[0]).to(device)
    means, ids, places, target, ends = [], [], [], [], [0]
    for n in counts:
        voxels, coords, filled = ssh.voxelize(cloud[:n].contiguous(), p.range_, p.cell, p.grid,
                                              p.max_points, p.max_voxels)
        means.append(voxels.sum(1) / filled[:, None])
        ids.append(coords[:, 1] * p.grid[0] + coords[:, 2])
        places.append(coords[:, 1:])
        target.append(filled.float() / p.max_points)
        ends.append(ends[-1] + coords.shape[0])
    means = torch.nan_to_num(torch.cat(means))
    scale = means.abs().amax(0).clamp(min=1e-6)
    return (means / scale, torch.cat(ids), torch.cat(places).contiguous(),
            torch.tensor(ends, dtype=torch.int32, device=device)), torch.cat(target), p


def main(steps=30, device="cuda"):
    torch.manual_seed(0)
    inputs, target, p = frames_of(device)
    model = PillarTokens(p.grid[0] * p.grid[1]).to(device)
    optimizer = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        found, _ = model(*inputs)
        loss = torch.nn.functional.mse_loss(found, target)
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
    with torch.no_grad():
        _, kept = model(*inputs)
    means, ids, places, offsets = inputs
    frames = offsets.shape[0] - 1
    last = offsets[1:].long() - 1  # asks again at each frame's last pillar
    answer, state = model.ask(model.features(means[last]), places[last].contiguous(), kept, offsets,
                              places)
    assert answer.shape == (frames,) and state.shape == (frames, model.width)
    return [float(v) for v in losses], answer.tolist()


def main_next(steps=30, device="cuda"):
    torch.manual_seed(0)
    inputs, _, p = frames_of(device)
    _, ids, _, offsets = inputs
    last = offsets[1:].long() - 1
    following = ids.roll(-1)
    following[last] = -1                # what follows a frame's last pillar is not known
    model = NextPillar(p.grid[0] * p.grid[1]).to(device)
    optimizer = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        x, _ = model(*inputs)
        loss = model.loss(x, following).sum() / (following >= 0).sum()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
    with torch.no_grad():
        # each frame but its last pillar, then that pillar alone from the kept states
        frames = offsets.shape[0] - 1
        kept = torch.ones(ids.shape[0], dtype=torch.bool, device=device)
        kept[last] = False
        ends = offsets - torch.arange(frames + 1, dtype=torch.int32, device=device)
        _, state = model(*(t[kept] for t in inputs[:3]), ends)
        one = torch.arange(frames + 1, dtype=torch.int32, device=device)
        x, _ = model(*(t[last] for t in inputs[:3]), one, state)
        answer = model.loss(x, ids[last])   # as likely as the same cell once more
    return [float(v) for v in losses], answer.tolist(), model


if __name__ == "__main__":
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 30
    losses, answer = main_next(steps)[:2] if sys.argv[2:] == ["next"] else main(steps)
    print("loss", " ".join(f"{v:.4f}" for v in losses[:3]), "...", f"{losses[-1]:.4f}")
    print("answers", " ".join(f"{v:.3f}" for v in answer))
