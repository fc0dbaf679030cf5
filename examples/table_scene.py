"""Trains a scene whose SH rows come from a shared table.

N Gaussians hold an index each into a table of V rows of SH coefficients (the
compact form of a scene: 4 N + 12 K V bytes of colour instead of 12 K N).  A
step looks the rows up, renders one view with its gradient, sums the
Gaussians' gradient rows into the table's gradient, forms the global norm of
the whole gradient and updates geometry and table with the clipped one, all on
the device and without a synchronisation beyond the view's own.

    python examples/table_scene.py [--gaussians N] [--rows V] [--steps S]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import differentiable_gaussian_splatting_amd as dgs  # noqa: E402
from differentiable_gaussian_splatting_amd import scenes  # noqa: E402


class TableScene:
    """A scene of the given geometry whose SH rows are table[index]; the table
    has its own moments beside the geometry's."""

    def __init__(self, ctx, scene, rows, seed=0):
        self.ctx = ctx
        self.ds = dgs.DeviceScene(scene, ctx.device)
        self.n, self.width = self.ds.n, 3 * (self.ds.sh_degree + 1) ** 2
        gen = torch.Generator().manual_seed(seed)
        self.index = torch.randint(0, rows, (self.n,), generator=gen, dtype=torch.int32).to(ctx.device)
        self.table = (0.2 * torch.randn((rows, self.width), generator=gen)).to(ctx.device)
        self.dtable = torch.zeros_like(self.table)
        # one gradient row per Gaussian: mean 3, log-scale 3, quaternion 4, opacity logit 1, SH
        self.rows = torch.zeros((self.n, 11 + self.width), device=ctx.device)
        self.sh = self.ds.sh.view(self.n, self.width)
        params = [self.ds.means, self.ds.log_scales, self.ds.quats, self.ds.logits.view(self.n, 1), self.table]
        columns = [self.rows[:, a:b] for a, b in ((0, 3), (3, 6), (6, 10), (10, 11))]
        zeros = lambda: [torch.zeros_like(p) for p in params]
        self.params, self.m, self.v = (dgs.TensorList(x) for x in (params, zeros(), zeros()))
        self.grads = dgs.TensorList(columns + [self.dtable])
        self.norm = torch.zeros(2, device=ctx.device)
        self.loss = torch.zeros(1, dtype=torch.float64, device=ctx.device)
        self.steps = 0

    def step(self, camera, target, lr=5e-3, max_norm=1e-3):
        """One view; its loss stays on the device (self.loss)."""
        ctx = self.ctx
        self.steps += 1
        dgs.gs_embed_fwd(ctx, self.table, self.index, self.sh)
        dgs.gs_train_view(ctx, camera, self.ds, target, grad3d_out=self.rows, loss_out=self.loss)
        dgs.gs_embed_bwd(ctx, self.index, self.rows[:, 11:], self.dtable)
        dgs.gs_grad_norm(ctx, self.grads, max_norm, self.norm)
        dgs.gs_adam_tensors(ctx, self.params, self.m, self.v, self.grads, step=self.steps, lr=lr, norm=self.norm)
        return self.loss


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--gaussians", type=int, default=20000)
    ap.add_argument("--rows", type=int, default=256)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--width", type=int, default=640)
    ap.add_argument("--height", type=int, default=400)
    a = ap.parse_args()
    ctx = dgs.Context()
    w = scenes.make_workload("c3_gmm4k", n=a.gaussians, width=a.width, height=a.height, seed=7)
    # the target: the scene with its own SH rows
    target = torch.zeros((3, a.height, a.width), device=ctx.device)
    dgs.gs_train_view(ctx, w.camera, dgs.DeviceScene(w.scene, ctx.device), torch.zeros_like(target), image_out=target)
    scene = TableScene(ctx, w.scene, a.rows)
    losses = []
    for _ in range(a.steps):
        losses.append(float(scene.step(w.camera, target)))
        if len(losses) % 10 == 1 or len(losses) == a.steps:
            norm, factor = scene.norm.tolist()
            print(f"step {len(losses):4d}  loss {losses[-1]:.6f}  gradient norm {norm:.4g}  factor {factor:.4g}", flush=True)
    ctx.close()
    return losses


if __name__ == "__main__":
    main()
