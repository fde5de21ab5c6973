"""Plans that share their rotation: made, closed and made again in any order and from several threads,
each keeps giving what its own signs and factors ask for."""
import threading

import numpy as np
import pytest

import kvgen
import oracle
from tests.parity import check_encode, check_rel_l2

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
FORMS = [(D, G, xf, bits) for D in (128, 256) for G in (32, 16) for xf in ("srft", "srht") for bits in (4, 8)]


@pytest.fixture(scope="module")
def kvq():
    import rotated_int4_kv_b200 as k
    return k


def use(kvq, plan, params, form, seed):
    """Encode and decode a few rows; both against the formula (wide factors, to tell plans apart)."""
    D, G, xf, bits = form
    x = np.random.default_rng(seed).standard_normal((1, 2, 40, D)).astype(np.float16)
    codes = torch.zeros((1, 2, 40, D * bits // 8), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1, 2, 40, D // G), dtype=torch.float16, device="cuda")
    kvq.encode(plan, torch.from_numpy(x).cuda(), codes, scales)
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    check_encode(x, *params, G, c, s, count_only=True, transform=xf, bits=bits, label=str(form))
    back = kvq.decode(plan, codes, scales, 0, 40).cpu().numpy().astype(np.float64)
    check_rel_l2(back.reshape(-1, D), oracle.decode(c, s, *params, G, xf, bits).reshape(-1, D), label=str(form))


def params_of(D, seed):
    signs, lam = kvgen.plan_params(D, seed=seed, kind="k")
    return signs, (lam * np.exp(0.5 * np.random.default_rng(seed).standard_normal(D))).astype(np.float32)


def test_plans_in_any_order(kvq):
    rng = np.random.default_rng(0)
    live = []
    for step in range(120):
        if live and rng.random() < 0.45:
            plan, params, form = live.pop(rng.integers(len(live)))
            use(kvq, plan, params, form, step)
            plan.close()
        else:
            form = FORMS[rng.integers(len(FORMS))]
            params = params_of(form[0], step)
            live.append((kvq.Plan(*params, form[1], form[2], form[3]), params, form))
    for plan, params, form in live:
        use(kvq, plan, params, form, 1)


def test_plans_made_by_several_threads(kvq):
    errors = []

    def work(k):
        try:
            torch.cuda.set_device(0)
            for i in range(25):
                form = FORMS[(k + i) % len(FORMS)]
                params = params_of(form[0], 100 * k + i)
                plan = kvq.Plan(*params, form[1], form[2], form[3])
                if i % 5 == 0:
                    use(kvq, plan, params, form, i)
                plan.close()
        except Exception as e:  # noqa: BLE001  (reported by the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
