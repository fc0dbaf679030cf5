"""A scene with SH rows from a table, end to end, and clipping inside a view."""
import os
import sys

import numpy as np
import pytest

from differentiable_gaussian_splatting_amd import binding as B
from differentiable_gaussian_splatting_amd import scenes
from tests.gpu_pipeline import rel_l2

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ctx():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    c = B.Context()
    yield c
    c.close()


def test_table_scene_learns(ctx):
    """The loss falls, the looked-up rows are the table's, and the table's
    gradient is the sum of its Gaussians' gradient rows."""
    import torch
    from table_scene import TableScene
    w = scenes.make_workload("c3_gmm4k", n=3000, width=160, height=96, seed=7)
    target = torch.zeros((3, 96, 160), device=ctx.device)
    B.gs_train_view(ctx, w.camera, B.DeviceScene(w.scene), torch.zeros_like(target), image_out=target)
    s = TableScene(ctx, w.scene, rows=37)
    losses = [float(s.step(w.camera, target)) for _ in range(40)]
    assert all(np.isfinite(losses)) and losses[-1] < 0.8 * losses[0], (losses[0], losses[-1])
    before = s.table.clone()
    s.step(w.camera, target)
    assert torch.equal(s.sh, before[s.index.long()])
    want = np.zeros((37, s.width))
    mags = np.zeros((37, s.width))
    g = s.rows[:, 11:].double().cpu().numpy()
    np.add.at(want, s.index.cpu().numpy(), g)
    np.add.at(mags, s.index.cpu().numpy(), np.abs(g))
    assert (np.abs(s.dtable.double().cpu().numpy() - want) <= 3000 * 2.0 ** -24 * mags + 1e-30).all()


def test_view_clips_its_gradient(ctx):
    """clip_norm scales the view's gradient to the norm, before grad3d_out and
    the update; the unclipped view is untouched by norm_out."""
    import torch
    w = scenes.make_workload("c2_hd", n=4000, width=200, height=120, posed=True, seed=12)
    target = torch.from_numpy(w.target).cuda()
    n, F = 4000, 59

    def view(clip, norm_out, budget=0):
        ds = B.DeviceScene(w.scene)
        m, v = B.like_scene(ds), B.like_scene(ds)
        g3 = torch.full((n, F), float("nan"), device="cuda")
        r = B.gs_train_view(ctx, w.camera, ds, target, loss="l1", budget_bytes=budget, grad3d_out=g3,
                            adam=dict(step=1, params=ds, m=m, v=v, lr=1e-3), clip_norm=clip, norm_out=norm_out)
        return r, g3, m, ds

    norm = torch.zeros(2, device="cuda")
    r0, g0, m0, _ = view(0.0, None)
    r1, g1, m1, _ = view(0.0, norm)
    true = float(g0.double().pow(2).sum().sqrt())
    # gradients of two runs differ by the order of the raster's atomic sums (1e-6 relative)
    assert abs(float(norm[0]) - true) <= 1e-4 * true and float(norm[1]) == 1.0
    assert rel_l2(g1.cpu().numpy(), g0.cpu().numpy()) <= 1e-4
    for budget in (0, 1_200_000):
        r2, g2, m2, _ = view(0.25 * true, norm, budget)
        assert abs(float(norm[0]) - true) <= 1e-4 * true and abs(float(norm[1]) - 0.25) <= 1e-4
        assert abs(r2["loss"] - r0["loss"]) <= 1e-6
        assert rel_l2(g2.cpu().numpy(), 0.25 * g0.cpu().numpy()) <= 2e-4
        # a first step's first moment is a tenth of the gradient it used
        assert rel_l2(m2.sh.cpu().numpy().reshape(n, -1), 0.1 * g2[:, 11:].cpu().numpy()) <= 1e-5
        assert rel_l2(m2.means.cpu().numpy(), 0.1 * g2[:, :3].cpu().numpy()) <= 1e-5
    # without outputs of its own: the clipped update alone
    ds = B.DeviceScene(w.scene)
    m, v = B.like_scene(ds), B.like_scene(ds)
    B.gs_train_view(ctx, w.camera, ds, target, loss="l1", adam=dict(step=1, params=ds, m=m, v=v), clip_norm=0.25 * true)
    assert rel_l2(m.sh.cpu().numpy().reshape(n, -1), 0.025 * g0[:, 11:].cpu().numpy()) <= 2e-4
    for bad in (-1.0, float("nan")):
        with pytest.raises(B.GsError) as e:
            B.gs_train_view(ctx, w.camera, ds, target, clip_norm=bad)
        assert e.value.status == B.GS_ERR_INVALID_ARG


def test_a_view_without_candidates_has_norm_zero(ctx):
    import torch
    w = scenes.make_workload("c1_small", n=50, width=32, height=32, seed=2)
    w.scene.means[:, 2] = -5.0
    norm = torch.full((2,), 7.0, device="cuda")
    ds = B.DeviceScene(w.scene)
    B.gs_train_view(ctx, w.camera, ds, torch.from_numpy(w.target).cuda(), clip_norm=1.0, norm_out=norm)
    assert norm.tolist() == [0.0, 1.0]


def test_a_clipped_view_that_cannot_allocate_changes_nothing():
    import torch
    from tests.test_gpu_errors import FailingContext
    f = FailingContext()
    w = scenes.make_workload("c1_small", n=300, width=64, height=48, seed=3, sh_degree=1)
    target = torch.from_numpy(w.target).cuda()
    ds = B.DeviceScene(w.scene)
    m, v = B.like_scene(ds), B.like_scene(ds)
    old = [t.clone() for t in ds.tensors()]
    live, k = f.mem_stats()["live"], 1
    while True:
        f.arm(k)
        try:
            B.gs_train_view(f, w.camera, ds, target, adam=dict(step=1, params=ds, m=m, v=v), clip_norm=1e-3)
            break
        except B.GsError as e:
            assert e.status == B.GS_ERR_OOM
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(old, ds.tensors()))
            assert all(float(t.abs().max()) == 0.0 for t in m.tensors() + v.tensors())
            assert f.mem_stats()["live"] == live
        k += 1
    f.arm(0)
    torch.cuda.synchronize()
    assert k > 3 and f.mem_stats()["live"] == live and not torch.equal(old[0], ds.means)
    f.close()


def _broken_view(ctx, **kw):
    """A first update of a view whose gradient is not finite for some of its Gaussians (a pixel of the target is
    NaN); returns the scene's tensors before and after, the moments, and the dense gradient."""
    import torch
    w = scenes.make_workload("c2_hd", n=4000, width=200, height=120, posed=True, seed=12)
    target = torch.from_numpy(w.target).cuda()
    target[:, 40, 60] = float("nan")
    ds = B.DeviceScene(w.scene)
    m, v = B.like_scene(ds), B.like_scene(ds)
    old = [t.clone() for t in ds.tensors()]
    g3 = torch.zeros((4000, 59), device="cuda")
    B.gs_train_view(ctx, w.camera, ds, target, loss="l1_ssim", grad3d_out=g3,
                    adam=dict(step=1, params=ds, m=m, v=v, lr=1e-3), **kw)
    return old, ds.tensors(), m.tensors() + v.tensors(), g3


def test_asking_for_the_norm_leaves_a_view_as_it_is(ctx):
    """norm_out without clip_norm scales nothing, also where a Gaussian's gradient is not finite: its neighbours
    are updated as without norm_out."""
    import torch
    _, new0, _, g0 = _broken_view(ctx)
    bad = ~g0.isfinite()
    assert 0 < int(bad.sum()) < bad.numel() // 2
    norm = torch.zeros(2, device="cuda")
    _, new1, _, g1 = _broken_view(ctx, norm_out=norm)
    assert torch.equal(~g1.isfinite(), bad)
    assert rel_l2(g1[~bad].cpu().numpy(), g0[~bad].cpu().numpy()) <= 1e-4
    for a, b in zip(new0, new1):
        assert torch.equal(a.isfinite(), b.isfinite())
    assert not norm.isfinite().any()


def test_clipped_view_leaves_an_update_out_whose_norm_is_not_finite(ctx):
    import torch
    for norm in (torch.zeros(2, device="cuda"), None):
        old, new, moments, _ = _broken_view(ctx, clip_norm=1.0, norm_out=norm)
        for a, b in zip(old, new):
            assert torch.equal(a, b)
        for t in moments:
            assert t.eq(0.0).all()
        assert norm is None or not norm[0].isfinite()


def test_a_view_that_the_gate_skips_has_norm_zero(ctx):
    """A gate runs the backward of some views of a sequence and skips others: norm and factor are those of
    this view, never of one before it."""
    import torch
    w = scenes.make_workload("c1_small", n=300, width=64, height=48, seed=3, sh_degree=1)
    target = torch.from_numpy(w.target).cuda()
    ds = B.DeviceScene(w.scene)
    gate = B.Gate(1, warmup=1)
    seen = set()
    for k, f in enumerate([1.0, 1.3, 0.7, 0.6, 1.4, 0.5, 0.45, 0.4]):
        norm = torch.full((2,), 7.0, device="cuda")
        r = B.gs_train_view(ctx, w.camera, ds, target * f, gate=gate, gate_view=0, clip_norm=1e-3, norm_out=norm)
        seen.add(r["backward"])
        if r["backward"]:
            assert norm[0] > 0.0 and norm[1] <= 1.0 and float(norm[0]) != 7.0
        else:
            assert norm.tolist() == [0.0, 1.0], k
    assert seen == {True, False}
    gate.close()
