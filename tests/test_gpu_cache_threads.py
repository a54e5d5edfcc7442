"""Host threads that attend with one cache on one stream."""
import threading

import pytest
import torch

from test_gpu_cache import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(dim=576, queries=16), dict(heads=2, queries=8, dim=64)])
def test_threads_on_one_stream_get_their_own_results(kw):
    """Two threads with different shapes and lengths alternate as they like; each call's results are
    those of the same call alone, bit for bit."""
    case = Case(98, [2500, 100, 1700], **kw)
    calls = [(case.q, case.dlen, case.dtable), (case.q[:1], case.dlen[1:2], case.dtable[1:2]),
             (case.q[1:], case.dlen[1:], case.dtable[1:])]
    alone = [case.cache.attend(0, *c, scale=0.1) for c in calls]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[] for _ in calls]

    def work(i):
        for _ in range(150):
            got[i].append(case.cache.attend(0, *calls[i], scale=0.1, stream=stream))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    case.cache.check()
    for one, all_of in zip(alone, got):
        assert len(all_of) == 150
        for out, lse in all_of:
            assert torch.equal(out, one[0]) and torch.equal(lse, one[1])
