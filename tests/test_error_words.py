"""The error words of step plans: each is given out once, whichever threads ask (no GPU needed)."""
import sys
import threading

import pytest

from sub_bit_moe_amd import api

torch = pytest.importorskip("torch")


def test_threads_of_one_stream_get_words_of_their_own(monkeypatch):
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda n, dtype, device: zeros(n, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(api, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(api, "_error_words", {})
    got = [[] for _ in range(4)]

    def ask(mine):
        for _ in range(20000):
            mine.append(api._error_word(0))

    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=ask, args=(mine,)) for mine in got]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    words = [w for mine in got for w in mine]
    assert all(w.numel() == 1 for w in words)
    assert len({w.data_ptr() for w in words}) == len(words) == 80000
