#!/usr/bin/env python3
"""A small message-passing potential, trained on the energies and forces of synthetic structures.

    python examples/train_energy.py [--steps 40] [--atoms 400] [--channels 32] [--lmax 2]

One training step runs the package's operators as a model uses them:

    species -> embed                       node features [N, C]
    conv_tp  (scalars in, degrees out)     block 1
    norm_residual                          r1 = r0 + alpha gate N(h1), u1 = N(r1)
    conv_tp  (degrees in, degrees out)     block 2
    norm_residual                          r2, u2; the scalars of u2 give the energies
    forces = -dE/d(edge vectors), summed onto atoms (first gradients, kept for the loss)
    backward of the energy and force loss, clip_grad_norm, one step of Adam

The radial weights of every edge come from a small torch network on Bessel
functions of the distance.  The targets are a number per species for every
atom and a repulsion exp(-distance) between neighbours.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import tensor_product_message_amd as ctp  # noqa: E402

SPECIES = 10
CUTOFF = 4.0


def structures(n_atoms, n_structures, device, seed):
    """Random atoms in boxes of 12 Angstrom, edges within the cutoff, receivers in order; energies and forces."""
    gen = torch.Generator().manual_seed(seed)
    pos = torch.rand(n_atoms, 3, generator=gen) * 12.0
    batch = torch.arange(n_atoms) * n_structures // n_atoms
    species = torch.randint(0, SPECIES, (n_atoms,), generator=gen, dtype=torch.int32)
    near = (torch.cdist(pos, pos) < CUTOFF) & (batch[:, None] == batch[None]) & ~torch.eye(n_atoms, dtype=torch.bool)
    recv, send = near.nonzero(as_tuple=True)
    row_ptr = torch.zeros(n_atoms + 1, dtype=torch.int32)
    row_ptr[1:] = torch.cumsum(near.sum(1), 0)
    of_species = torch.randn(SPECIES, generator=gen)
    vec = pos[recv] - pos[send]
    pair = torch.exp(-vec.norm(dim=1))
    energy = torch.zeros(n_structures).index_add_(0, batch, of_species[species.long()])
    energy.index_add_(0, batch[recv], 0.5 * pair)
    forces = torch.zeros(n_atoms, 3).index_add_(0, recv, pair[:, None] * vec / vec.norm(dim=1, keepdim=True))
    graph = ctp.Graph(n_atoms, row_ptr.to(device), send.to(torch.int32).to(device))
    edges = (recv.to(device), send.to(device))
    return species.to(device), vec.to(device), edges, graph, batch.to(device), energy.to(device), forces.to(device)


class Potential(torch.nn.Module):
    def __init__(self, channels, lmax, device):
        super().__init__()
        self.lmax, self.channels = lmax, channels
        new = lambda *shape, std=1.0, mean=0.0: torch.nn.Parameter(  # noqa: E731
            torch.randn(shape, device=device) * std + mean)
        self.table = new(SPECIES, channels)
        self.paths = [ctp.num_paths(0, lmax, lmax), ctp.num_paths(lmax)]
        self.radial = torch.nn.ModuleList(
            torch.nn.Sequential(torch.nn.Linear(8, 32), torch.nn.SiLU(), torch.nn.Linear(32, p * channels)).to(device)
            for p in self.paths)
        self.w_post = torch.nn.ParameterList(new(lmax + 1, channels, std=0.0, mean=1.0) for _ in range(2))
        self.w_pre = torch.nn.ParameterList(new(lmax + 1, channels, std=0.0, mean=1.0) for _ in range(2))
        self.gate = torch.nn.ParameterList(new(lmax + 1, channels, std=0.1, mean=0.5) for _ in range(2))
        self.readout = new(channels, std=channels ** -0.5)

    def forward(self, species, vec, graph, batch, n_structures):
        L, C, n = self.lmax, self.channels, species.numel()
        dist = vec.norm(dim=1, keepdim=True)
        k = torch.arange(1, 9, device=vec.device) * math.pi / CUTOFF
        bessel = torch.sin(k * dist) / dist * (1 + torch.cos(math.pi * dist / CUTOFF)) / 2
        w = [net(bessel).view(-1, p, C) for net, p in zip(self.radial, self.paths)]
        x = ctp.embed(self.table, species)                              # [N, C]
        r = torch.cat([x[:, None], x.new_zeros(n, (L + 1) ** 2 - 1, C)], 1)
        h = ctp.conv_tp(x[:, None], vec, w[0], graph, (0, L, L), ctp.VEC_GIVEN)
        r, u = ctp.norm_residual(h, r, self.w_post[0], self.w_pre[0], self.gate[0], alpha=0.5, lmax=L)
        h = ctp.conv_tp(u, vec, w[1], graph, L, ctp.VEC_GIVEN)
        r, u = ctp.norm_residual(h, r, self.w_post[1], self.w_pre[1], self.gate[1], alpha=0.5, lmax=L)
        return u.new_zeros(n_structures).index_add(0, batch, u[:, 0] @ self.readout)


def train(steps=40, atoms=400, channels=32, lmax=2, n_structures=8, max_norm=10.0, seed=0, device="cuda:0", log=print):
    """(losses, gradient norms) of every step, as lists."""
    torch.manual_seed(seed)
    species, vec, (recv, send), graph, batch, energy, forces = structures(atoms, n_structures, torch.device(device), seed)
    vec.requires_grad_()
    model = Potential(channels, lmax, device)
    params = list(model.parameters())
    adam = torch.optim.Adam(params, lr=1e-2)
    losses, norms = [], []
    per_atom = atoms / n_structures
    for step in range(steps):
        adam.zero_grad()
        e = model(species, vec, graph, batch, n_structures)
        g, = torch.autograd.grad(e.sum(), vec, create_graph=True)
        f = torch.zeros_like(forces).index_add(0, send, g).index_add(0, recv, -g)
        loss = ((e - energy) / per_atom).square().mean() + (f - forces).square().mean()
        loss.backward(inputs=params)
        grads = [p.grad for p in params]
        _, norm = ctp.clip_grad_norm(grads, max_norm, out=grads)
        adam.step()
        losses.append(loss.detach())
        norms.append(norm)
        if log and step % 10 == 0:
            log(f"step {step:4d}  loss {float(losses[-1]):.5f}  gradient norm {float(norm):.3f}")
    return [float(x) for x in losses], [float(x) for x in norms]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("steps", 40), ("atoms", 400), ("channels", 32), ("lmax", 2)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    losses, _ = train(a.steps, a.atoms, a.channels, a.lmax)
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f}")
