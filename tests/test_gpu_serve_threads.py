"""Other Python threads run while a single-token call waits."""
import threading
import time

import pytest
import torch

from tests.test_gpu_serve import kda  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["step", "cache_append", "cache_attend"])
def test_a_call_that_waits_lets_others_run(kda, name):  # noqa: F811
    """Calls behind half a second of work fill the queue of launches, and the next one waits for room there: a thread
    that ticks every millisecond goes on ticking."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    kc, vc = kda.new_cache(4, 16, 2, 64, 64)
    table, lens = z(2, 2, dt=torch.int32), z(2, dt=torch.int32)
    heads, out, ws = z(2, 2, 64), z(2, 2, 64), z(1 << 16, dt=torch.uint8)
    token, state = z(2, 1, 2, 64), z(2, 2, 64, 64, dt=torch.float32)
    g, beta, o = token.float(), token[..., 0].contiguous(), token.clone()
    call = dict(step=lambda: kda.step(token, token, token, g, beta, state, out=o),
                cache_append=lambda: kda.cache_append(heads, heads, kc, vc, table, lens, q=heads, q_out=out),
                cache_attend=lambda: kda.cache_attend(heads, kc, vc, table, lens, out=out, ws=ws))[name]
    call()
    torch.cuda.synchronize()
    ticks, done = [], threading.Event()

    def tick():
        while not done.is_set():
            ticks.append(time.perf_counter())
            time.sleep(1e-3)

    other = threading.Thread(target=tick)
    other.start()
    try:
        longest = 0.0
        torch.cuda._sleep(1_000_000_000)  # about half a second
        end = time.perf_counter() + 0.3
        while time.perf_counter() < end:
            began = time.perf_counter()
            call()
            longest = max(longest, time.perf_counter() - began)
        torch.cuda.synchronize()
    finally:
        done.set()
        other.join()
    assert longest > 0.2  # (the case is the one that it is meant to be)
    assert max(b - a for a, b in zip(ticks, ticks[1:])) < 0.1
