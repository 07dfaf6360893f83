"""prefill without max_q_len reads the offsets on the stream that it is given: they may be written there just
before."""

import pytest
import torch

import attn_cases as A
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


def test_offsets_written_on_the_given_stream_just_before():
    c = A.make("bf16", [300, 70, 200], [40, 3, 130], 8, 2, 128, seed=9)
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    lens = torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
    ready = torch.tensor([0, 40, 43, 173], dtype=torch.int32, device="cuda")
    starts = torch.zeros_like(ready)  # what the current stream sees: no rows at all
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms of the stream's work before
        starts.copy_(ready)
    got = pa.prefill(dev["q"], dev["k"], dev["v"], dev["table"], lens, starts, c["scale"], stream=side)
    torch.cuda.synchronize()
    assert pa.check_device_errors() == pa.PA_OK
    A.check(c, "prefill", got)
