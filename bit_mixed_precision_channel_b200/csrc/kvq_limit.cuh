// kvq_limit.cuh — a limit that is only ever raised, by any number of threads (host code).
#pragma once
#include <pthread.h>

namespace kvq {

// Calls set(value), which returns 0 on success, unless `seen` says that a value at least as
// large was set before.  The attribute and its record change together under the lock: with a
// bare record, a smaller value set between a larger one's call and its record would lower the
// attribute for good while the record kept the larger.  (Plain pthreads: nothing here throws.)
template <typename Set>
inline int raise_limit(int& seen, int value, Set set) {
  if (value <= __atomic_load_n(&seen, __ATOMIC_ACQUIRE)) return 0;
  static pthread_mutex_t mutex = PTHREAD_MUTEX_INITIALIZER;
  pthread_mutex_lock(&mutex);
  int e = 0;
  if (value > __atomic_load_n(&seen, __ATOMIC_ACQUIRE)) {
    e = set(value);
    if (e == 0) __atomic_store_n(&seen, value, __ATOMIC_RELEASE);
  }
  pthread_mutex_unlock(&mutex);
  return e;
}

}  // namespace kvq
