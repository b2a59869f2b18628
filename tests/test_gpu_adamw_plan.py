"""The lifetime of an AdamW plan's tensors on other streams than their own."""
import pytest

from tests.gpu_util import announce, torch_cuda
from tests.test_gpu_adamw_tensors import B1, B2, EPS, LR, _tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["argument", "context"])
@pytest.mark.parametrize("bits", [32, 8])
def test_dropped_plan_keeps_its_memory_until_the_step_has_run(how, bits):
    """The plan is the last to hold its tensors and is dropped while the step still
    waits in a side stream: new tensors of the same sizes get other memory."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("dropped plan", how, bits)
    n = 3 << 20         # (a size that nothing else here has)
    ts = _tensors(torch, [n], "f32", "bf16", bits)
    kept = ts[0]["p"]
    before = kept.clone()
    mine = [v for v in ts[0].values() if isinstance(v, torch.Tensor)]
    plan = qlin.qlin_adamw_tensors_plan(ts)
    taken = {t.untyped_storage().data_ptr() for t in [*mine, plan.image]}
    like = [(t.shape, t.dtype) for t in [*mine[1:], plan.image]]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)      # (a tenth of a second or so)
    if how == "argument":
        qlin.qlin_adamw_tensors(plan, LR, B1, B2, EPS, 1, 1, stream=side)
    else:
        with torch.cuda.stream(side):
            qlin.qlin_adamw_tensors(plan, LR, B1, B2, EPS, 1, 1)
    del plan, ts, mine
    fresh = [torch.empty(s, dtype=d, device="cuda") for s, d in like]
    assert not side.query()                 # the step had not run yet
    assert not taken & {t.untyped_storage().data_ptr() for t in fresh}
    side.synchronize()
    assert (kept != before).float().mean() > 0.9


def test_steps_on_one_stream_record_it_once():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    plan = qlin.qlin_adamw_tensors_plan(_tensors(torch, [100, 3000], "f32", "f32", 32))
    side = torch.cuda.Stream()
    for step in range(1, 6):
        qlin.qlin_adamw_tensors(plan, LR, B1, B2, EPS, 1, step)
        qlin.qlin_adamw_tensors(plan, LR, B1, B2, EPS, 1, step, stream=side)
    assert len(plan._streams) == 2
    torch.cuda.synchronize()
