"""Inline loads from shared memory that ordinary C++ stores have written: the compiler orders
them only if the statement says that it reads memory (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_quantized_gemm_q4_gb300", "csrc")
TOUCHES = re.compile(r"\b(ld|st)\.(shared|global)|\b(ldmatrix|cp\.async|atom|red|bar|barrier|mbarrier)\b")


def statements(text):
    """Each asm statement: its instructions and all of it."""
    for m in re.finditer(r"\basm(\s+volatile)?\s*\(", text):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            quoted ^= c == '"' and text[at - 1] != "\\"
            depth += 0 if quoted else (c == "(") - (c == ")")
            at += 1
        body = text[m.end():at - 1]
        yield "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body.split(":", 1)[0])) or body, m.group(0) + body


def test_statements():
    got = list(statements('asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(f(a)) : "memory"); asm("add.s32 %0;" : "=r"(x));'))
    assert [g[0] for g in got] == ["ld.shared.b32 %0, [%1];", "add.s32 %0;"] and '"memory"' in got[0][1] and '"memory"' not in got[1][1]


@pytest.mark.parametrize("name", ["kv_attention.cu", "kv_attention.cuh", "kv_attention_rows.cu", "kv_append_rotary.cu", "lora.cu"])
def test_memory_is_named(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    found = [(code, full) for code, full in statements(text) if TOUCHES.search(code)]
    assert found or name == "kv_append_rotary.cu"
    assert [code for code, full in found if "volatile" not in full or '"memory"' not in full] == []
