"""What an AdamWPlan keeps: its table's memory while steps on other streams still read it, and the
tensors that the table points to.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


def test_a_dropped_plan_keeps_its_table_for_a_step_on_another_stream(P):
    """A plan of one stream, stepped on another that is behind other work and dropped at once: its table's
    memory is not handed out on the first stream before that step has run, and the step is the usual one."""
    n = 200_000
    p, g = torch.randn(n, device=DEV), torch.randn(n, device=DEV)
    want = P.AdamWTensor.new(p.clone(), g, 32)
    P.adamw_step(P.AdamWPlan([want]), lr=1e-3, step=1)
    t = P.AdamWTensor.new(p.clone(), g, 32)
    plan = P.AdamWPlan([t])
    at, size = plan.table.data_ptr(), plan.table.numel()
    side = torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(200):
            busy = torch.mm(busy, busy).mul_(1e-2)
        P.adamw_step(plan, lr=1e-3, step=1)
    del plan
    taken = [torch.empty(size, dtype=torch.int64, device=DEV) for _ in range(8)]
    assert not side.query(), "the step had already run"
    assert at not in [x.data_ptr() for x in taken]
    torch.cuda.synchronize()
    assert torch.equal(t.param, want.param) and torch.equal(t.v, want.v)


def test_a_replaced_tensor_needs_another_plan(P):
    """A field set anew after the plan was built is refused, not left unread, until it is set back or
    planned again; other plans go on, and what the table points to stays allocated."""
    n = 4096
    a, b = (P.AdamWTensor.new(torch.randn(n, device=DEV), torch.randn(n, device=DEV), 32) for _ in range(2))
    plan, other = P.AdamWPlan([a]), P.AdamWPlan([b])
    P.adamw_step(plan, lr=1e-3, step=1)
    was, at = a.grad, a.grad.data_ptr()
    a.grad = torch.randn(n, device=DEV)
    before = a.param.clone()
    for _ in range(2):
        with pytest.raises(P.PmnError, match=r"tensors\[0\].grad"):
            P.adamw_step(plan, lr=1e-3, step=2)
    P.adamw_step(other, lr=1e-3, step=1)
    assert torch.equal(a.param, before)
    ref = P.AdamWTensor(before.clone(), a.grad, a.m.clone(), a.v.clone())
    P.adamw_step(P.AdamWPlan([a]), lr=1e-3, step=2)
    P.adamw_step(P.AdamWPlan([ref]), lr=1e-3, step=2)
    assert torch.equal(a.param, ref.param)
    fresh, a.grad = a.grad, was
    P.adamw_step(plan, lr=1e-3, step=3)
    a.weight_decay = 0.5
    with pytest.raises(P.PmnError, match="weight_decay"):
        P.adamw_step(plan, lr=1e-3, step=4)
    a.weight_decay = 0.0 * n
    P.adamw_step(plan, lr=1e-3, step=4)
    a.grad = fresh
    del was
    torch.cuda.synchronize()
    assert at not in [torch.empty(n, device=DEV).data_ptr() for _ in range(4)]


def test_the_norms_gradient_goes_to_the_planned_buffer(P):
    """dgamma written where the plan reads it, over several steps and in a replayed graph: the same weights
    as with the gradient copied there."""
    rows, cols = 300, 520
    z = torch.randn((rows, cols), device=DEV).to(torch.bfloat16)
    dy = torch.randn((rows, cols), device=DEV).to(torch.bfloat16)

    def program(copied):
        gamma, grad = torch.ones(cols, device=DEV), torch.zeros(cols, device=DEV)
        plan = P.AdamWPlan([P.AdamWTensor.new(gamma, grad, 32)])
        count = torch.ones(1, dtype=torch.int64, device=DEV)

        def step():
            o = P.rmsnorm_residual_fwd(z, gamma, want_rstd=True)
            if copied:
                grad.copy_(P.rmsnorm_residual_bwd(dy, z, gamma, o.rstd)[1])
            else:
                assert P.rmsnorm_residual_bwd(dy, z, gamma, o.rstd, dgamma=grad)[1] is grad
            P.adamw_step(plan, lr=1e-2, step=count)
            count.add_(1)
        return step, gamma

    (by_copy, a), (given, b), (captured, c) = program(True), program(False), program(False)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured()
    for _ in range(3):
        by_copy()
        given()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(a, c) and not (a == 1).any()
    buf = torch.empty(cols + 8, device=DEV).fill_(7.0)
    P.rmsnorm_residual_bwd(z[:0], z[:0], a, torch.empty(0, device=DEV), dgamma=buf[4:-4])
    assert (buf[4:-4] == 0).all() and (buf[:4] == 7).all() and (buf[-4:] == 7).all()
