"""Kept plans under threads: those of the Python forms are the module's, and a server's threads meet there."""
import copy
import pickle
import sys
import threading

import pytest

from structured_sparse_gemm_nm_amd import feed_forward


@pytest.fixture
def switches():
    was = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    yield
    sys.setswitchinterval(was)


def test_threads_with_ever_new_plans(switches, monkeypatch):
    monkeypatch.setattr(feed_forward, "MOST_PLANS", 3)
    plans, wrong = feed_forward._Plans(), []

    def work(first):
        try:
            for i in range(30000):
                key = (first + i) % 11
                if plans.get(key, lambda: [key])[0] != key:
                    wrong.append(key)
        except Exception as e:                          # noqa: BLE001 - whatever it is, the test names it
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(3 * t,)) for t in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
    assert len(plans) <= 3


def test_a_copy_has_plans_of_its_own():
    plans = feed_forward._Plans()
    kept = plans.get(1, object)
    for other in (copy.deepcopy(plans), copy.copy(plans), pickle.loads(pickle.dumps(plans))):
        assert len(other) == 0 and other.get(1, object) is not kept and plans.get(1, object) is kept
