"""Routing and distillation without a GPU: the entry points before sim_init,
and the 64-bit oracle of their GPU tests against automatic differentiation
and the formulas' own identities."""
import pytest
import torch

from tests import loss_oracle as oracle


def test_refused_before_init():
    import all_reduce_reduction_amd as sim
    sim.sim_finalize()
    assert sim.sim_route(None, 8, "bf16", None, 0, 8, 2, 1, None, None, None, None, None, 0) == -9
    assert sim.sim_route_grad(None, 8, "bf16", None, 0, 8, 2, 1, None, None, None, None, 0.0, None, 8, None) == -9
    assert sim.sim_distill_step(None, 8, "bf16", 0, 8, None, None, "fp32", 2, 1.0, None, 1.0, None, 8, None, None,
                                0) == -9
    assert sim.sim_distill_parts(None, 8, "bf16", 0, 8, 0, 8, None, None, "fp32", 2, 1.0, None, None, 0) == -9
    assert sim.sim_distill_join(None, 1, 0, 8, None, None, "fp32", 2, 1.0, None, None) == -9
    assert sim.sim_distill_grad(None, 8, "bf16", 0, 8, 0, 8, None, None, "fp32", 2, 1.0, None, None, 1.0, None, 8) == -9
    for f in (lambda: sim.sim_route_work(1, 8, 2, "bf16"), lambda: sim.sim_distill_work(1, 8, "bf16")):
        with pytest.raises(sim.SimError):
            f()


def test_helpers_refuse_host_tensors():
    import all_reduce_reduction_amd as sim
    x, i, z = torch.zeros(2, 8), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    with pytest.raises(ValueError):
        sim.route(x, 2)
    with pytest.raises(ValueError):
        sim.route_grad(x, i)
    with pytest.raises(ValueError):
        sim.distill_step(x, i, z)
    with pytest.raises(ValueError):
        sim.distill_parts(x, i, z)
    with pytest.raises(ValueError):
        sim.distill_grad(x, i, z, torch.zeros(2, 2))


def test_limits_match_the_header():
    import os
    import re

    import all_reduce_reduction_amd as sim
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "simar.h")).read()
    for name in ("ROUTE_MAX_EXPERTS", "ROUTE_MAX_TOPK", "DISTILL_MAX_TOPK"):
        assert getattr(sim, name) == int(re.search(rf"#define SIM_{name} (\d+)", text).group(1))


@pytest.mark.parametrize("normalize", [False, True])
def test_route_gradient_is_that_of_the_objective(normalize):
    g = torch.Generator().manual_seed(1)
    t, e, k, coef = 7, 20, 4, 3.0
    x = torch.randn(t, e, generator=g, dtype=torch.float64, requires_grad=True)
    keep = torch.arange(t) != 3
    chosen, w, counts, sums, _, _ = oracle.route(x.detach(), k, keep, normalize)
    dw = torch.randn(t, k, generator=g)
    oracle.route_objective(x, chosen, dw, counts, coef, keep, normalize).backward()
    want, _ = oracle.route_grad(x.detach(), chosen, dw, counts, coef, keep, normalize)
    assert torch.allclose(x.grad, want, rtol=1e-12, atol=1e-14)
    # every kept row's probabilities sum to one, every kept row chooses k experts
    assert abs(sums.sum().item() - 6) < 1e-12 and counts[:e].sum() == 6 * k and counts[e] == 6
    if normalize:
        assert torch.allclose(w[keep].sum(1), torch.ones(6, dtype=torch.float64))


def test_even_routing_has_the_least_balance_loss():
    e, k = 8, 2
    counts = torch.tensor([5] * e + [20], dtype=torch.int32)
    even = oracle.balance_loss(None, counts, torch.full((e,), 20.0 / e), k, 1.0)
    assert abs(even.item() - 1.0) < 1e-12  # coef times one
    skew = oracle.balance_loss(None, torch.tensor([20, 20] + [0] * (e - 2) + [20], dtype=torch.int32),
                               torch.tensor([10.0, 10.0] + [0.0] * (e - 2)), k, 1.0)
    assert skew.item() > even.item()


def test_distillation_gradient_is_that_of_the_loss():
    g = torch.Generator().manual_seed(2)
    t, v, k, tau = 6, 40, 5, 1.7
    x = torch.randn(t, v, generator=g, dtype=torch.float64, requires_grad=True)
    ids = torch.randint(-2, v, (t, k), generator=g, dtype=torch.int32)
    ids[4] = -1
    z = torch.randn(t, k, generator=g)
    scale = torch.rand(t, generator=g)
    (oracle.distill_loss(x, ids, z, tau) * scale.double()).sum().backward()
    loss, _, d, _ = oracle.distill(x.detach(), ids, z, tau, scale, 1.0)
    assert torch.allclose(x.grad, d, rtol=1e-12, atol=1e-14)
    assert loss[4] == 0 and not d[4].any() and (loss >= 0).all()


def test_a_student_equal_to_its_teacher_has_no_loss():
    z = torch.randn(3, 6, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    x = torch.full((3, 50), -torch.inf, dtype=torch.float64)
    ids = torch.arange(10, 16, dtype=torch.int32).expand(3, 6).contiguous()
    x.scatter_(1, ids.long(), z)
    loss, _, d, _ = oracle.distill(x, ids, z, 1.0, None, 1.0)
    assert loss.abs().max() < 1e-12 and d.abs().max() < 1e-12
