"""fa_get_device_status synchronises with the device: it reports what calls on any stream met,
also on streams that do not wait for the default one."""
import pytest
import torch

import exact_io_aware_27_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


def test_status_of_a_call_still_queued_on_another_stream():
    bad = torch.tensor([0, 3, 1], dtype=torch.int32, device="cuda")
    fa.fa_packed_plan(bad, 4)
    assert fa.fa_get_device_status() == -8
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # some 0.1 s
    plan = fa.fa_packed_plan(bad, 4, stream=side)
    assert fa.fa_get_device_status() == -8
    assert side.query()
    assert fa.fa_get_device_status() == 0
    assert plan.nseq == 2
