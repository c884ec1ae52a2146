// The functions of csrc/kv4_counts.cuh for the CPU tests (tests/test_kv4_counts.py).
#include "kv4_counts.cuh"

extern "C" {

int count_words() { return spark::kCountWords; }

void first_count(int from, int to, int *out) {
    const spark::StateCount c = spark::kv4_first_count(from, to);
    out[0] = c.word, out[1] = c.shift, out[2] = c.bits;
}

void second_count(int c0, int *out) {
    const spark::StateCount c = spark::kv4_second_count(c0);
    out[0] = c.word, out[1] = c.shift, out[2] = c.bits;
}

void group(int c0, int c1, int cta, int *out) {
    const spark::StateGroup g = spark::kv4_group(c0, c1, cta);
    out[0] = g.from, out[1] = g.to, out[2] = g.groups;
}

}  // extern "C"
