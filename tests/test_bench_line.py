"""The bench's table of configuration points: every figure of every point, in a line of a length that is read."""
import json
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import bench  # noqa: E402


def point(i, oracle=True):
    names = ["decode_step_graph_us", "decode_step_fused_graph_us", "merged_us", "attn2_us", "topk_us", "gather_us",
             "quantize_us", "merged_hbm_frac", "attn2_hbm_frac", "quantize_hbm_frac", "gather_gbs"]
    pt = {"B": 4, "N": 131072, "bits": 2, "group": 32, "k": 5243, "low_bit_bytes_per_token": 96,
          "decode_step_fused_launches": 3, "merged_bytes": 490389504, "gather_bytes": 85901312}
    pt.update({n: 1000.0 * math.pi / (i + j + 1) for j, n in enumerate(names)})
    if oracle:
        pt.update(oracle_ms_per_layer=7635.9321600000385 + i, oracle_pairs=1, layer_pairs=32, oracle_threads=1)
    return pt


def measured():
    res = {n: {"workload": "a layer of some shape, B=8, 32/8 heads, N=32768, 1-bit, k=328", "points": [point(i)]}
           for i, n in enumerate(("c1", "c2", "c3", "g64_1bit", "g64_2bit"))}
    res["c3"] = {"workload": "one that failed", "error": "RuntimeError: why"}
    pts = [point(i, oracle=i != 7) for i in range(48)]
    pts[5] = {"B": 1, "N": 4096, "bits": 1, "error": "RuntimeError: why"}
    res["c5"] = {"workload": "48 points", "points": pts}
    return res


def test_every_figure_is_in_the_table():
    res = measured()
    out = json.loads(json.dumps(bench.configs_table(res)))
    assert out["c3"] == res["c3"]
    for name, cfg in res.items():
        assert out[name]["workload"] == cfg["workload"]
        for pt, row in zip(cfg.get("points", []), out[name].get("points", []), strict=True):
            got = dict(zip(out["columns"], row, strict=True))
            for key, x in pt.items():
                assert got[key] == x or abs(got[key] - x) <= 5e-5 * abs(x)
            assert all(got[key] is None for key in got if key not in pt)
    assert bench.configs_table(None) is None


def test_the_table_is_short():
    """The rest of the line is about 6 KB."""
    assert len(json.dumps(bench.configs_table(measured()))) < 14000
