"""Calls from several host threads at once, a stream and a scratch each: launches
of one kernel instance with more and with less shared memory."""

import threading

import pytest
import torch

import paged_split_kv_02_gb300 as pd
from paged_split_kv_02_gb300 import workloads as W
from gpu_helpers import scratch_for
from step_cases import run_sinks

pytestmark = pytest.mark.gpu


def test_calls_of_many_sizes_from_several_threads():
    pd.build()
    pd.paged_decode_device_status(reset=True)
    cases, want = [], []
    for k, S in enumerate((30, 900, 60, 400)):
        c = W.make_case("threads", seed=k, dtype=torch.bfloat16, head_size=64, num_q_heads=8 * (k + 1),
                        num_kv_heads=8, page_size=16, max_query_len=1 + k, seq_lens=[40 + k] * S, window=20)
        cases.append(c.to("cuda"))
        want.append(run_sinks(cases[k], 4, scratch_for(c, 16)))
    torch.cuda.synchronize()
    failed = []

    def work(k):
        try:
            st, sc = torch.cuda.Stream(), scratch_for(cases[k], 16)
            outs = [torch.empty_like(cases[k].q) for _ in range(40)]
            torch.cuda.synchronize()
            for o in outs:
                run_sinks(cases[k], 4, sc, out=o, stream=st)
            st.synchronize()
            if not all(torch.equal(o, want[k]) for o in outs):
                failed.append((k, "outputs"))
        except Exception as e:  # a thread's own errors do not reach the test
            failed.append((k, e))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert pd.paged_decode_device_status(reset=True) == 0
