"""attention_4bit called from several host threads on one stream: a call's
kernels use the stream's workspace, so no other call's may come between them."""
import threading
import time

import pytest
import torch

from quantized_matvec_amd import attention, attention_4bit
from test_gpu_attention import make

pytestmark = pytest.mark.gpu


class Slow:
    """The library with an enqueue that takes a while, as one that waits for a
    full queue does, and that notes which workspaces are in use meanwhile."""

    def __init__(self, lib):
        self._lib, self._used, self.shared, self.calls = lib, [], 0, 0

    def __getattr__(self, name):
        return getattr(self._lib, name)

    def qmv_attention_4bit(self, *args):
        key = (args[-1], args[-3])      # stream, workspace
        self.calls += 1
        self.shared += key in self._used
        self._used.append(key)
        time.sleep(0.02)
        rc = self._lib.qmv_attention_4bit(*args)
        self._used.remove(key)
        return rc


def test_calls_on_one_stream_do_not_share_a_workspace_at_once(monkeypatch):
    cache, table, _, _ = make([9000, 700], 2, 128, 64, 16, "bf16", "nf4", 51)
    kl = torch.tensor([9000, 700], dtype=torch.int32, device="cuda")
    qs = [torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16) for _ in range(4)]
    want = [attention_4bit(q, cache, table, kl) for q in qs]
    torch.cuda.synchronize()
    slow = Slow(attention.lib())
    monkeypatch.setattr(attention, "lib", lambda: slow)
    got = [[] for _ in qs]

    def work(i):
        for _ in range(5):
            got[i].append(attention_4bit(qs[i], cache, table, kl))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(qs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert slow.calls == 20 and slow.shared == 0
    for g, w in zip(got, want):
        assert len(g) == 5 and all(torch.equal(x, w) for x in g)


def test_many_threads_get_their_own_results():
    """Decode and divided prompts, on the default stream and on streams of their own."""
    cache, table, _, _ = make([20000, 300], 2, 64, 64, 64, "bf16", "nf4", 52)
    kl = torch.tensor([20000, 300], dtype=torch.int32, device="cuda")
    cus = [None, torch.tensor([0, 40, 64], dtype=torch.int32, device="cuda")]
    qs = [torch.randn(2 if i % 2 == 0 else 64, 4, 64, device="cuda").to(torch.bfloat16) for i in range(8)]
    call = lambda i: attention_4bit(qs[i], cache, table, kl, cu_q=cus[i % 2], max_q=1 if i % 2 == 0 else 40)
    want = [call(i) for i in range(8)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream() if i % 4 == 3 else torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            outs = [call(i) for _ in range(200)]
        stream.synchronize()
        wrong.extend(i for o in outs if not torch.equal(o, want[i]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
