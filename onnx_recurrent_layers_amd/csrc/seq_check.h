// seq_check.h -- what the C ABI of the operators beside the recurrent layers
// shares: checked sizes, scratch regions, the tensors of a call, the stream's
// device.  Internal.
#pragma once

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "seq_ops.h"

namespace rnnhip {

constexpr int64_t kMaxBytes = int64_t(1) << 52;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;   // of one launch

inline int fail(int code, const char* who, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_error_of(code, who, buf);
}

// a*b*c*... in bytes, or -1 when it overflows the largest tensor accepted.
inline int64_t bytes_of(std::initializer_list<int64_t> f) {
  int64_t n = 1;
  for (int64_t x : f) {
    if (x < 0) return -1;
    if (x == 0) return 0;
  }
  for (int64_t x : f) {
    if (n > kMaxBytes / x) return -1;
    n *= x;
  }
  return n;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int elem_size(int dtype) { return dtype == RNN_DTYPE_F32 ? 4 : 2; }

// Scratch regions, 256-byte aligned.
struct Regions {
  size_t off = 0;
  bool ok = true;
  size_t take(std::initializer_list<int64_t> f) {
    const int64_t n = bytes_of(f);
    const size_t at = off;
    if (n < 0 || off > size_t(kMaxBytes)) ok = false;
    else off = (off + size_t(n) + 255) & ~size_t(255);
    return at;
  }
};

// The stream's device for the time of a call.
class OnDevice {
 public:
  explicit OnDevice(hipStream_t s) {
    if (!s || s == hipStreamPerThread) return;
    hipDevice_t d = 0;
    int cur = 0;
    if (hipStreamGetDevice(s, &d) != hipSuccess || hipGetDevice(&cur) != hipSuccess || cur == int(d)) return;
    if (hipSetDevice(int(d)) == hipSuccess) back_ = cur;
  }
  ~OnDevice() {
    if (back_ >= 0) (void)hipSetDevice(back_);
  }

 private:
  int back_ = -1;
};

// The tensors of one call: resolved one by one, the first failure kept.
class Tensors {
 public:
  explicit Tensors(const char* who) : who_(who) {}
  int status = RNN_OK;

  char* tensor(const rnn_tensor& t, int es, const char* name, bool required, bool output = false) {
    return resolve(t.ptr, t.elem_offset, es, name, required, output);
  }
  Rows rows(const rnn_rows& t, int es, int64_t length, int64_t count, const char* name, bool required, bool output = false) {
    Rows r{nullptr, length};
    if (status != RNN_OK) return r;
    if (t.ptr) {
      if (t.row_stride != 0 && t.row_stride < length) {
        status = fail(RNN_ERR_SHAPE, who_, "%s: row_stride %lld below the row's length %lld", name, (long long)t.row_stride,
                      (long long)length);
        return r;
      }
      if (t.row_stride) r.rs = t.row_stride;
      if (bytes_of({std::max<int64_t>(count, 1), r.rs, es}) < 0) {
        status = fail(RNN_ERR_SHAPE, who_, "%s: size overflows", name);
        return r;
      }
    }
    r.p = resolve(t.ptr, t.elem_offset, es, name, required, output);
    return r;
  }
  // An output may share its first element with no other tensor of the call;
  // each pair names two that may be one buffer, in the order that they are resolved.
  struct Pair {
    const char *a, *b;
  };
  void apart(std::initializer_list<Pair> pairs = {}) {
    for (int i = 0; i < n_ && status == RNN_OK; ++i)
      for (int j = 0; j < i && status == RNN_OK; ++j)
        if (seen_[i].p == seen_[j].p && (seen_[i].output || seen_[j].output) &&
            std::none_of(pairs.begin(), pairs.end(), [&](const Pair& p) { return !std::strcmp(seen_[i].name, p.b) && !std::strcmp(seen_[j].name, p.a); }))
          status = fail(RNN_ERR_ARG, who_, "%s: the same memory as %s", seen_[i].name, seen_[j].name);
  }

 private:
  struct Seen {
    const char* p;
    const char* name;
    bool output;
  };
  const char* who_;
  Seen seen_[32];
  int n_ = 0;

  char* resolve(void* ptr, int64_t offset, int es, const char* name, bool required, bool output) {
    if (status != RNN_OK) return nullptr;
    if (!ptr) {
      if (required) status = fail(RNN_ERR_ARG, who_, "%s: NULL", name);
      return nullptr;
    }
    if (offset < 0) {
      status = fail(RNN_ERR_ARG, who_, "%s: negative element offset", name);
      return nullptr;
    }
    if (offset > kMaxBytes / es) {
      status = fail(RNN_ERR_SHAPE, who_, "%s: element offset overflows", name);
      return nullptr;
    }
    char* p = static_cast<char*>(ptr) + offset * es;
    if (reinterpret_cast<uintptr_t>(p) % uintptr_t(es)) {
      status = fail(RNN_ERR_ARG, who_, "%s: address not aligned to its %d-byte element", name, es);
      return nullptr;
    }
    if (n_ < 32) seen_[n_++] = Seen{p, name, output};
    return p;
  }
};

inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool aligned(const Rows& r, size_t n, int es) { return aligned(r.p, n) && (size_t(r.rs) * size_t(es)) % n == 0; }

inline int check_scratch(const char* who, void* scratch, size_t need) {
  if (!need) return RNN_OK;
  if (!scratch) return fail(RNN_ERR_ARG, who, "scratch: NULL (needs %zu bytes)", need);
  if (!aligned(scratch, 256)) return fail(RNN_ERR_ARG, who, "scratch: not 256-byte aligned");
  return RNN_OK;
}

inline int check_seq(const char* who, int dtype, int direction, int layout, int64_t seq, int64_t batch, int64_t channels,
                     const char* name = "channels") {
  if (dtype < RNN_DTYPE_F32 || dtype > RNN_DTYPE_BF16) return fail(RNN_ERR_ARG, who, "dtype: unknown value %d", dtype);
  if (direction == RNN_DIR_BIDIRECTIONAL)
    return fail(RNN_ERR_ARG, who, "direction: forward or reverse (two problems for both)");
  if (direction != RNN_DIR_FORWARD && direction != RNN_DIR_REVERSE)
    return fail(RNN_ERR_ARG, who, "direction: unknown value %d", direction);
  if (layout != 0 && layout != 1) return fail(RNN_ERR_ARG, who, "layout: must be 0 or 1, got %d", layout);
  if (seq < 0) return fail(RNN_ERR_SHAPE, who, "seq: negative (%lld)", (long long)seq);
  if (batch < 0) return fail(RNN_ERR_SHAPE, who, "batch: negative (%lld)", (long long)batch);
  if (channels < 1) return fail(RNN_ERR_SHAPE, who, "%s: must be at least 1 (%lld)", name, (long long)channels);
  if (channels > (int64_t(1) << 24)) return fail(RNN_ERR_UNSUPPORTED, who, "%s: above 16777216", name);
  if (batch > (int64_t(1) << 30)) return fail(RNN_ERR_UNSUPPORTED, who, "batch: above 2^30");
  if (seq > (int64_t(1) << 30)) return fail(RNN_ERR_UNSUPPORTED, who, "seq: above 2^30");
  return RNN_OK;
}

inline SeqGeom geometry(int64_t seq, int64_t batch, int layout, int direction, const char* lens) {
  SeqGeom g;
  g.S = int(seq);
  g.B = int(batch);
  g.layout = layout;
  g.reverse = direction == RNN_DIR_REVERSE;
  g.lens = reinterpret_cast<const int32_t*>(lens);
  return g;
}

// Names that may be one buffer.
inline constexpr char kInitial[] = "initial_state", kFinal[] = "final_state";

}  // namespace rnnhip
